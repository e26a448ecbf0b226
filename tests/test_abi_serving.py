"""Host-side refusals of the ragged serving calls. CPU only: every call here returns before
anything is launched (addresses are made up and never read)."""
import ctypes

import numpy as np
import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 0x10000  # an address aligned to everything
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_13_gb300 import build
    build.build()
    from mla_latent_kv_13_gb300 import mla as m
    return m


def call(lib, name, order, good, **change):
    args = dict(good, **change)
    return getattr(lib, name)(*(args[k] for k in order))


def check(mla, name, order, good, refusals):
    lib = mla.lib()
    # nothing but the workspace is wrong with the good call
    assert call(lib, name, order, good, ws_bytes=0) == WORKSPACE
    for change, want in refusals:
        assert call(lib, name, order, good, **change) == want, change


CHUNK = ("q_lat q_rope kv num_blocks table max_blocks q_starts seqlens B tokens H max_seqlen "
         "window sinks scale ws ws_bytes out lse stream").split()
WINDOW = ("q_lat q_rope kv num_blocks table max_blocks seqlens B s_q H max_seqlen window sinks "
          "scale splits ws ws_bytes out lse stream").split()
ATTENTION = dict(q_lat=P, q_rope=P, kv=P, codes=P, exps=P, num_blocks=9, table=P, max_blocks=4,
                 q_starts=P, seqlens=P, B=2, tokens=5, s_q=1, H=16, max_seqlen=256, window=7,
                 sinks=0, scale=0.1, splits=0, ws=P, ws_bytes=1 << 40, out=P, lse=P, stream=None)
ATTENTION_REFUSALS = [
    *(({k: None}, INVALID) for k in ("q_lat", "q_rope", "table", "seqlens", "out", "lse", "ws")),
    ({"num_blocks": 0}, INVALID), ({"max_blocks": 0}, INVALID), ({"max_seqlen": 257}, INVALID),
    ({"max_seqlen": -1}, INVALID), ({"sinks": -1}, INVALID), ({"scale": 0.0}, INVALID),
    ({"scale": -1.0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"B": 0}, INVALID), ({"B": 4097}, INVALID),
    ({"H": 17}, UNSUPPORTED), ({"H": 0}, UNSUPPORTED), ({"H": 256}, UNSUPPORTED),
    ({"num_blocks": (1 << 24) + 1}, UNSUPPORTED), ({"q_lat": P + 8}, INVALID),
    ({"q_rope": P + 2}, INVALID), ({"out": P + 16}, INVALID), ({"lse": P + 2}, INVALID),
    ({"ws": P + 128}, INVALID), ({"table": P + 2}, INVALID),
]


def fp8(order):
    return [x for k in order for x in (("codes", "exps") if k == "kv" else (k,))]


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_chunk_attention(mla, cache):
    name, order = "mla_chunk_attention", CHUNK
    more = [({"kv": None}, INVALID), ({"kv": P + 4}, INVALID)]
    if cache == "fp8":
        name, order = name + "_fp8", fp8(order)
        more = [({"codes": None}, INVALID), ({"exps": None}, INVALID), ({"exps": P + 8}, INVALID)]
    check(mla, name, order, ATTENTION, ATTENTION_REFUSALS + more + [
        ({"q_starts": None}, INVALID), ({"tokens": 0}, INVALID), ({"window": -1}, INVALID),
        ({"tokens": (1 << 20) + 1}, UNSUPPORTED),
        # the schedule's weights would pass 32 bits
        ({"tokens": 1 << 20, "H": 128, "max_blocks": 1 << 20, "max_seqlen": 1 << 26,
          "window": 0}, UNSUPPORTED),
    ])


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_window_decode(mla, cache):
    name, order = "mla_decode_attention_window", WINDOW
    more = [({"kv": None}, INVALID)]
    if cache == "fp8":
        name, order = name + "_fp8", fp8(order)
        more = [({"codes": None}, INVALID), ({"exps": None}, INVALID)]
    check(mla, name, order, ATTENTION, ATTENTION_REFUSALS + more + [
        ({"s_q": 0}, INVALID), ({"s_q": 9}, UNSUPPORTED), ({"s_q": MAX}, UNSUPPORTED),
        ({"window": 0}, INVALID), ({"splits": -1}, INVALID), ({"splits": 257}, INVALID),
    ])


def test_attention_workspace_sizes(mla):
    size = mla.chunk_workspace_size
    assert size(3, 40, 16, 1000) >= size(3, 40, 16, 100) > mla.WS_HEADER_BYTES
    # a window bounds what an item can see, whatever the lengths
    assert size(2, 2, 16, 1 << 20, window=64) == size(2, 2, 16, 1 << 10, window=64)
    for bad in (dict(B=0), dict(tokens=0), dict(max_seqlen=-1), dict(window=-1), dict(sinks=-1)):
        with pytest.raises(mla.MLAError):
            size(**dict(dict(B=2, tokens=2, H=16, max_seqlen=9), **bad))
    assert mla.decode_window_workspace_size(2, 1, 128, MAX, MAX, MAX, 1) == mla.WS_HEADER_BYTES


NORM = ("x ldx q_lora w_q w_kv eps q_starts seqlens B tokens table max_blocks kv num_blocks theta "
        "c_q ws ws_bytes stream").split()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_norm_rope_append(mla, cache):
    good = dict(x=P, ldx=640, q_lora=64, w_q=P, w_kv=P, eps=1e-6, q_starts=P, seqlens=P, B=2,
                tokens=5, table=P, max_blocks=4, kv=P, codes=P, exps=P, num_blocks=9,
                theta=10000.0, c_q=P, ws=P, ws_bytes=256, stream=None)
    name, order = "mla_norm_rope_append", NORM
    caches = ("kv",)
    if cache == "fp8":
        name, order, caches = name + "_fp8", fp8(order), ("codes", "exps")
    check(mla, name, order, good, [
        *(({k: None}, INVALID) for k in ("x", "w_q", "w_kv", "q_starts", "seqlens", "table",
                                         "c_q", "ws", *caches)),
        ({"B": 0}, INVALID), ({"B": 4097}, INVALID), ({"tokens": 0}, INVALID),
        ({"q_lora": -8}, INVALID), ({"q_lora": 60}, INVALID), ({"ldx": 632}, INVALID),
        ({"ldx": 644}, INVALID), ({"max_blocks": 0}, INVALID), ({"num_blocks": 0}, INVALID),
        ({"eps": -1e-6}, INVALID), ({"eps": float("inf")}, INVALID), ({"theta": 0.0}, INVALID),
        ({"theta": float("nan")}, INVALID), ({"x": P + 8}, INVALID), ({"w_kv": P + 8}, INVALID),
        ({"c_q": P + 8}, INVALID), ({caches[0]: P + 8}, INVALID), ({"ws": P + 64}, INVALID),
        ({"max_blocks": 1 << 25}, UNSUPPORTED), ({"q_lora": 65544, "ldx": 1 << 20}, UNSUPPORTED),
    ])
    # without a query side its arrays may be absent
    assert call(mla.lib(), name, order, good, q_lora=0, ldx=576, w_q=None, c_q=None,
                ws_bytes=0) == WORKSPACE


def test_absorb_q_latent(mla):
    order = ("c_q B q_lora w_uq w_qr w_uk H pos theta ws ws_bytes q_lat q_rope stream").split()
    good = dict(c_q=P, B=2, q_lora=64, w_uq=P, w_qr=P, w_uk=P, H=16, pos=P, theta=10000.0, ws=P,
                ws_bytes=1 << 40, q_lat=P, q_rope=P, stream=None)
    check(mla, "mla_absorb_q_latent", order, good, [
        *(({k: None}, INVALID) for k in ("c_q", "w_uq", "w_qr", "w_uk", "pos", "ws", "q_lat",
                                         "q_rope")),
        ({"B": 0}, INVALID), ({"q_lora": 72}, INVALID), ({"H": 3}, UNSUPPORTED),
        ({"theta": -1.0}, INVALID), ({"c_q": P + 8}, INVALID), ({"ws": P + 16}, INVALID),
    ])


STATE = "refs num_blocks table max_blocks seqlens num_seqs".split()
PAGES = dict(refs=P, num_blocks=100, table=P, max_blocks=4, seqlens=P, num_seqs=9, rows=P, lens=P,
             parents=P, children=P, n=3, refs_out=P, table_out=P, live=P, ws=P, ws_bytes=1 << 40,
             stream=None)
PAGES_REFUSALS = [
    *(({k: None}, INVALID) for k in ("refs", "table", "seqlens", "ws")),
    ({"num_blocks": 0}, INVALID), ({"max_blocks": 0}, INVALID), ({"num_seqs": 0}, INVALID),
    ({"num_blocks": (1 << 24) + 1}, UNSUPPORTED), ({"num_seqs": (1 << 20) + 1}, UNSUPPORTED),
    ({"max_blocks": 1 << 25}, UNSUPPORTED), ({"refs": P + 2}, INVALID), ({"ws": P + 8}, INVALID),
]


def pool(mla, **kw):
    p = dict(base=P, page_bytes=73728, layer_stride=100 * 73728, layers=2)
    p.update(kw)
    return (mla._Pool * 1)(mla._Pool(p["base"], p["page_bytes"], p["layer_stride"], p["layers"]))


def test_pages(mla):
    lib, tail = mla.lib(), "ws ws_bytes stream".split()
    good = dict(PAGES, pools=pool(mla), n_pools=1)
    lists = {"mla_pages_free": ["rows"], "mla_pages_extend": ["rows", "lens"]}
    for name, arrays in lists.items():
        order = STATE + arrays + ["n"] + tail
        check(mla, name, order, good, PAGES_REFUSALS + [({"n": -1}, INVALID)] +
              [({a: None}, INVALID) for a in arrays])
        assert call(lib, name, order, good, n=0, **{a: None for a in arrays}) == 0
    fork = STATE + "parents children n pools n_pools".split() + tail
    compact = STATE + "refs_out table_out live pools n_pools".split() + tail
    pools = [({"pools": None}, INVALID), ({"n_pools": -1}, INVALID), ({"n_pools": 5}, INVALID)]
    for bad in (dict(base=None), dict(base=P + 8), dict(layers=0), dict(page_bytes=0),
                dict(page_bytes=24), dict(layer_stride=73728), dict(layer_stride=100 * 73728 + 8)):
        pools.append(({"pools": pool(mla, **bad)}, INVALID))
    check(mla, "mla_pages_fork", fork, good, PAGES_REFUSALS + pools + [
        ({"n": -1}, INVALID), ({"n": 4097}, UNSUPPORTED), ({"parents": None}, INVALID),
        ({"children": None}, INVALID)])
    assert call(lib, "mla_pages_extend", STATE + ["rows", "lens", "n"] + tail, good,
                n=4097) == UNSUPPORTED
    check(mla, "mla_pages_compact", compact, good, PAGES_REFUSALS + pools + [
        ({k: None}, INVALID) for k in ("refs_out", "table_out", "live")])


def test_status_name(mla):
    mla.lib().mla_status_string.restype = ctypes.c_char_p
    assert mla.lib().mla_status_string(7) == b"MLA_ERR_NO_PAGES" == mla.STATUS[7].encode()


def test_binding_checks_tensors(mla):
    import torch
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        mla._arg(t, mla._BF16, 2, 3)
    with pytest.raises(ValueError, match="shape"):
        mla._arg(t, mla._I32, 3, 2)
    with pytest.raises(ValueError, match="CUDA"):
        mla._arg(t, mla._I32, 2, 3)
    q = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.chunk_attention(q, q[..., :64], q, t, t[0], t[0, :2], 64, 0.1, out=q, lse=q, workspace=q)
    with pytest.raises(ValueError):
        mla.norm_rope_append(q[0], None, q[0, 0], t[0], t[0, :2], t, q)
    with pytest.raises(ValueError, match="pools"):
        mla._pools([torch.zeros(2, 5, 4)], 5)
    with pytest.raises(ValueError, match="at most"):
        mla._pools([t] * 5, 3)


def test_bf16_bits_are_nearest_even():
    # the tests' own rounding, against torch's
    import torch
    from tests import rows_ref
    x = np.random.default_rng(0).standard_normal(4096).astype(np.float32) * 1e3
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(rows_ref.bf16_bits(x), want)


def test_binding_refusals_without_a_device(mla):
    """What the compiled binding answers to wrong arguments: Python's errors, from every call."""
    import torch
    q = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(5, 64, 576, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    own = dict(out=q, lse=q, workspace=q)
    for call in (
            lambda: mla.chunk_attention(q, q, pages, table, i, i, 9, 0.1, **own),
            lambda: mla.chunk_attention(q[0], q, pages, table, i, i, 9, 0.1, **own),  # 2 dimensions
            lambda: mla.chunk_attention_fp8(q, q, pages, pages, table, i, i, 9, 0.1, **own),
            lambda: mla.decode_attention_window(q, q, pages, table, i, 9, 3, 0, 0.1, **own),
            lambda: mla.decode_attention_window(i, q, pages, table, i, 9, 3, 0, 0.1, **own),
            lambda: mla.decode_attention_window_fp8(q, q, i, i, table, i, 9, 3, 0, 0.1, **own),
            lambda: mla.norm_rope_append(i, i, i, i, i, table, pages, c_q=q, workspace=q),
            lambda: mla.pages_free(i, table, i, i, workspace=i),
            lambda: mla.pages_extend(table, table, i, i, i, workspace=i),
            lambda: mla.pages_fork(i, table, i, i, i, [pages], workspace=i),
            lambda: mla.pages_compact(i, table, i, [pages], live=i, workspace=i)):
        with pytest.raises((TypeError, ValueError)):
            call()
    for wrong in (None, 3, "q", [q], np.zeros(3)):  # not a tensor
        with pytest.raises(TypeError):
            mla.chunk_attention(wrong, q, pages, table, i, i, 9, 0.1, **own)
        with pytest.raises(TypeError):
            mla.pages_free(i, wrong, i, i, workspace=i)
    with pytest.raises(TypeError, match="bfloat16"):
        mla.chunk_attention(q.double(), q, pages, table, i, i, 9, 0.1, **own)
    with pytest.raises(TypeError, match="arguments"):
        mla._binding.chunk(q)
    with pytest.raises(TypeError):
        mla._pools(7, 3)


def test_binding_counts_no_references(mla):
    """Refused calls leave every argument's reference count as it was."""
    import sys
    import torch
    q = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    pools = [q, q]
    before = sys.getrefcount(q), sys.getrefcount(pools)
    for _ in range(100):
        with pytest.raises((TypeError, ValueError)):
            mla._pools(pools, 3)
        with pytest.raises((TypeError, ValueError)):
            mla.pages_free(q, q, q, q, workspace=q)
    after = sys.getrefcount(q), sys.getrefcount(pools)
    assert after == before


def test_a_window_workspace_serves_smaller_batches(mla):
    """What the largest shape wants is enough for every smaller one."""
    size = mla.decode_window_workspace_size
    base = dict(B=5, s_q=1, H=128, max_seqlen=9000, window=512, sinks=4)
    for heads, s_q in ((128, 1), (16, 3), (32, 4)):
        for name, values in (("B", [*range(1, 100), 500, 4096]),
                             ("max_seqlen", range(0, 12000, 64)),
                             ("window", range(1, 9000, 100)), ("sinks", range(0, 9000, 100))):
            for splits in (0, 1, 5):
                got = [size(**{**base, "H": heads, "s_q": s_q, "num_splits": splits, name: v})
                       for v in values]
                assert got == sorted(got), (heads, name, splits)
    for B in (1, 30, 64, 76, 77, 300):
        for splits in (0, 1, 3):
            got = [size(B, s, 16, 5000, 600, 4, splits) for s in range(1, 9)]
            assert got == sorted(got)
    # several arguments at once, against the largest shape of a server
    most = size(100, 4, 32, 8192, 1024, 64)
    rng = np.random.default_rng(0)
    for _ in range(300):
        assert size(int(rng.integers(1, 101)), int(rng.integers(1, 5)), 32,
                    int(rng.integers(0, 8193)), int(rng.integers(1, 1025)),
                    int(rng.integers(0, 65))) <= most
