"""Decode attention of batches that share prefixes, through the C ABI, against the plain 64-bit form
(tests/rows_ref.py says how the bounds come about)."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def shared_case(seed, heads, s_q, groups, lone=(), fp8=False, size=0.6):
    """Groups (prefix, lengths) one after another, then sequences of no group; pages in shuffled
    order, -1 behind each sequence's pages, NaN in every cached row that no token sees."""
    lens = [n for _, ns in groups for n in ns] + list(lone)
    d = R.attention_case(seed, heads, [s_q] * len(lens), lens, fp8=fp8, size=size)
    d["s_q"] = s_q
    starts, b = [0], 0
    for prefix, ns in groups:
        mine = range(b, b + len(ns))
        longest = max(mine, key=lambda i: lens[i])
        for i in mine:
            k = min(prefix // 64, lens[i] // 64)
            d["table"][i, :k] = d["table"][longest, :k]
        # a page that one sequence fills only in part and the group has in common is whole in the
        # longest one; the shorter one sees it in part
        b += len(ns)
        starts.append(b)
    d["groups"] = np.array(starts, np.int32)
    d["prefix"] = np.array([p for p, _ in groups], np.int32)
    return d


def run(mla, d, **kw):
    B, s_q, H = len(d["lens"]), d["s_q"], d["heads"]
    q = dev_bf16(d["q"])
    lead = (B, H) if s_q == 1 else (B, s_q, H)
    q_lat = q[..., :512].reshape(*lead, 512).contiguous()
    q_rope = q[..., 512:].reshape(*lead, 64).contiguous()
    if "codes" in d:
        call = mla.decode_attention_shared_fp8
        cache = (torch.from_numpy(d["codes"]).cuda(), torch.from_numpy(d["exps"]).cuda())
    else:
        call, cache = mla.decode_attention_shared, (dev_bf16(d["bits"]),)
    out, lse, ws = call(q_lat, q_rope, *cache, dev_i32(d["table"]), dev_i32(d["lens"]),
                        dev_i32(d["groups"]), dev_i32(d["prefix"]), d.get("most", max(d["lens"])),
                        d["scale"], **kw)
    assert out.shape == (*lead, 512) and lse.shape == lead
    return out.reshape(B * s_q, H, 512), lse.reshape(B * s_q, H), mla.check_device_status(ws)


def check(d, out, lse, status=0):
    assert status == 0
    ref, lref, tol, ltol = R.attention(d)
    # the merge of parts: each is off by no more than what was rounded in it, and the sums over the
    # parts (under 64 of them, fp32) by 64 * 2^-23 of the sum of magnitudes, which is within 1e-5
    R.assert_within(lse.cpu().numpy().astype(np.float64), lref, ltol + 1e-5, "lse")
    got = torch.from_numpy(host_bits(out).astype(np.int32) << 16).view(torch.float32).double().numpy()
    R.assert_within(got, ref, tol + 1e-5 * np.abs(ref).max(), "out")


GROUPS = {
    "one group": ([(1300, [1301, 1500, 1300, 1364, 1400, 1311, 1999, 1302, 1500])], ()),
    "two groups and lone ones": ([(640, [700] * 9), (900, [901, 960, 1024, 1100, 902])], (5, 300)),
    "nothing in common": ([(0, [70, 9]), (63, [64, 65, 90])], ()),
    "prefix beyond all": ([(10 ** 6, [500, 700, 300, 64, 65, 1, 900, 900])], ()),
    "shorter than the prefix": ([(1280, [1, 64, 1400, 700, 65, 127, 128, 129, 1281])], ()),
    "empty ones": ([(640, [0, 900, 0, 0, 641, 700, 0, 650, 800, 900, 641]), (64, [0, 0])], (0, 3)),
    "one of each": ([(700, [800]), (700, [701]), (128, [200, 129])], ()),
    "no tail": ([(1024, [1024] * 8)], ()),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("heads,s_q", [(16, 1), (16, 3), (16, 8), (32, 1), (32, 2), (64, 1), (64, 2),
                                       (128, 1)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_shared(mla, name, heads, s_q, fp8):
    groups, lone = GROUPS[name]
    d = shared_case(1, heads, s_q, groups, lone, fp8=fp8)
    check(d, *run(mla, d))


LONG = {
    # (heads, tokens, groups, lone): items cut into many parts, and few-part items beside them
    "one of 128 heads": (128, 1, [(0, [8000])], ()),
    "eight samples": (16, 1, [(9000, [9001 + 130 * i for i in range(8)])], ()),
    "48 rows": (16, 3, [(7000, [7777])], ()),
    "80 rows and empty ones": (16, 5, [(0, [0]), (0, [4500]), (0, [0])], (6001, 0)),
    "two of many parts, five of few": (128, 1, [(4000, [4001, 4800])], (300, 1, 65, 129, 640)),
    "the largest item of all clusters": (128, 1, [(0, [10113])], ()),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("name", list(LONG))
def test_long_items(mla, name, fp8):
    """Items in up to a part for each of 76 clusters: the sums over parts are off by 76 * 2^-23 = 9.1e-6
    of the magnitudes, still within check's 1e-5."""
    heads, s_q, groups, lone = LONG[name]
    d = shared_case(9, heads, s_q, groups, lone, fp8=fp8)
    check(d, *run(mla, d))


@pytest.mark.parametrize("heads", [16, 64])
def test_many_groups(mla, heads):
    rng = np.random.default_rng(5)
    groups = []
    for _ in range(40):
        p = int(rng.integers(1, 900))
        groups.append((p, [p + int(rng.integers(1, 200)) for _ in range(rng.integers(1, 12))]))
    d = shared_case(2, heads, 1, groups)
    check(d, *run(mla, d))


def test_larger_bounds_and_workspace(mla):
    """A bound far above the lengths and a workspace for a larger batch."""
    d = shared_case(3, 32, 1, [(1000, [1001, 1200, 1300, 1010, 1020])])
    d["most"] = d["table"].shape[1] * 64
    ws = mla.alloc_workspace(mla.decode_shared_workspace_size(64, 1, 32, 20000, 7))
    check(d, *run(mla, d, workspace=ws))


def test_as_plain_decode(mla):
    """The same batch without groups' help: mla_decode_attention over the same tables."""
    d = shared_case(4, 64, 1, [(1900, [1950, 2000, 2100, 1901, 1999, 2048])])
    out, lse, status = run(mla, d)
    q = dev_bf16(d["q"])
    want, wlse, ws = mla.decode_attention(q[..., :512].contiguous(), q[..., 512:].contiguous(),
                                          dev_bf16(d["bits"]), dev_i32(d["table"]),
                                          dev_i32(d["lens"]), max(d["lens"]), d["scale"])
    assert status == 0 and mla.check_device_status(ws) == 0
    # both are within half a step and a little of the same value
    assert torch.allclose(lse, wlse, atol=1e-4, rtol=0)
    assert (out.double() - want.double()).norm() <= 2 ** -7 * want.double().norm()


def test_common_pages_are_read_once(mla):
    """The shared pages come out of the longest sequence's table: the others' entries are not read
    where the group is large enough to share."""
    d = shared_case(6, 16, 1, [(2560, [2561 + 40 * i for i in range(8)])])
    ref = run(mla, d)
    d["table"][:7, :40] = -7
    got = run(mla, d)
    assert got[2] == 0 and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_what_is_recorded(mla):
    groups = [(640, [700, 800, 900, 650, 1000, 641, 642, 643])]
    d = shared_case(7, 16, 1, groups)
    # ranges that do not ascend: nothing is shared, and everything still right
    for bad in ([0, 9], [-1, 8], [5, 3]):
        d["groups"] = np.array(bad, np.int32)
        out, lse, status = run(mla, d)
        assert status == 4
        check(d, out, lse)
    d["groups"] = np.array([0, 8], np.int32)
    d["prefix"] = np.array([-5], np.int32)
    out, lse, status = run(mla, d)
    assert status == 4
    check(d, out, lse)
    # a page id out of the pool, in the common part and in a tail: masked as a page of no rows
    d = shared_case(7, 16, 1, groups)
    longest = 4
    d["table"][longest, 2] = d["pool"]
    d["table"][1, 12] = -3
    out, lse, status = run(mla, d)
    assert status == 4
    for b, n in enumerate(d["lens"]):
        j = np.arange(n)
        gone = (j // 64 == 2) | ((b == 1) & (j // 64 == 12))
        page = np.where(j // 64 < 10, d["table"][longest, j // 64], d["table"][b, j // 64])
        kv = d["cache"][page[~gone], j[~gone] % 64]
        q = torch.from_numpy((d["q"][b].astype(np.int32) << 16)).view(torch.float32).double().numpy()
        s = d["scale"] * q @ kv.T
        w = np.exp(s - s.max(1, keepdims=True))
        want = (w / w.sum(1, keepdims=True)) @ kv[:, :512]
        got = out[b].double().cpu().numpy()
        # half a step of the weights and one of the output, of values up to about 1
        assert np.abs(got - want).max() <= 2 ** -6 * max(1, np.abs(want).max())
    # lengths out of range are clamped
    d = shared_case(8, 16, 1, groups)
    d["most"] = 1000
    lens = list(d["lens"])
    d["lens"] = [n if i != 4 else 5000 for i, n in enumerate(lens)]
    out, lse, status = run(mla, d)
    assert status == 4
    d["lens"] = lens
    check(d, out, lse)


def test_replayed_graph(mla):
    """One captured call serves other lengths, groups and tables of the same sizes."""
    ds = [shared_case(10, 16, 2, [(1280, [1300 + 30 * i for i in range(9)]), (300, [400, 500, 310])]),
          shared_case(11, 16, 2, [(64, [90, 100]), (700, [0, 3, 800, 701, 900, 720, 730, 740, 750, 760])])]
    blocks = max(d["table"].shape[1] for d in ds)
    pool = max(d["pool"] for d in ds)
    B, H, most = 12, 16, blocks * 64

    def tensors(d):
        table = np.full((B, blocks), -1, np.int32)
        table[:, :d["table"].shape[1]] = d["table"]
        bits = np.zeros((pool, 64, 576), np.uint16)
        bits[:d["pool"]] = d["bits"]
        q = dev_bf16(d["q"]).reshape(B, 2, H, 576)
        return [q[..., :512].contiguous(), q[..., 512:].contiguous(), dev_bf16(bits), dev_i32(table),
                dev_i32(d["lens"]), dev_i32(d["groups"]), dev_i32(d["prefix"])]

    held = tensors(ds[0])
    out = torch.empty(B, 2, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, 2, H, device="cuda")
    ws = mla.alloc_workspace(mla.decode_shared_workspace_size(B, 2, H, most, 2))
    call = lambda: mla.decode_attention_shared(*held, most, R.SCALE, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for d in (ds[1], ds[0], ds[1]):
        for to, t in zip(held, tensors(d)):
            to.copy_(t)
        out.fill_(7), lse.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert mla.check_device_status(ws) == 0
        check(d, out.reshape(B * 2, H, 512), lse.reshape(B * 2, H))
        first = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)  # no order of atomics shows


def test_own_stream(mla):
    d = shared_case(12, 32, 1, [(2000, [2001 + 9 * i for i in range(12)])])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    out, lse, status = run(mla, d, stream=st)
    st.synchronize()
    check(d, out, lse, status)


def test_refused(mla):
    d = shared_case(13, 16, 1, [(64, [100, 200])])
    with pytest.raises(ValueError):
        run(mla, dict(d, prefix=np.zeros(3, np.int32)))
    with pytest.raises(mla.MLAError):
        run(mla, d, workspace=mla.alloc_workspace(0))
    with pytest.raises(mla.MLAError):
        run(mla, dict(d, scale=-1.0))
    with pytest.raises(mla.MLAError):
        run(mla, dict(d, most=10 ** 6))


def test_nothing_cached(mla):
    """A batch of empty sequences, with a bound of no rows at all too."""
    for most in (0, 64):
        d = shared_case(14, 32, 1, [(100, [0, 0, 0]), (0, [0])])
        d["most"] = most
        check(d, *run(mla, d))


@pytest.mark.parametrize("batch", [600, 4096])
def test_large_batches(mla, batch):
    """More sequences than one round of the list's threads, in many groups and in one."""
    rng = np.random.default_rng(15)
    for size in (7, batch):
        groups = []
        for b in range(0, batch, size):
            p = int(rng.integers(0, 200))
            groups.append((p, [int(p + rng.integers(0, 3)) if rng.random() < 0.97 else 0
                               for _ in range(min(size, batch - b))]))
        d = shared_case(15, 16, 1, groups)
        out, lse, status = run(mla, d)
        assert status == 0
        only = set(rng.choice(batch, 100, replace=False).tolist()) | {0, batch - 1}
        ref, lref, tol, ltol = R.attention(d, only)
        at = sorted(only)
        R.assert_within(lse.cpu().numpy().astype(np.float64)[at], lref[at], ltol[at] + 1e-5, "lse")
        got = torch.from_numpy(host_bits(out).astype(np.int32) << 16).view(torch.float32).double().numpy()
        R.assert_within(got[at], ref[at], tol[at] + 1e-5 * np.abs(ref).max(), "out")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_far_pages(mla, fp8):
    """Pages whose bytes lie behind 2^32 of the cache's start."""
    d = shared_case(16, 16, 1, [(700, [701, 800, 900, 1000, 720, 730, 740, 750])], fp8=fp8)
    pool = 130000 if fp8 else 70000
    move = np.random.default_rng(16).permutation(pool)[:d["pool"]]
    move[:4] = [pool - 1, pool - 2, 0, pool // 2]
    move = np.unique(move)[:d["pool"]]
    while len(move) < d["pool"]:
        move = np.append(move, np.setdiff1d(np.arange(1000), move)[0])
    big = dict(d, pool=pool, table=np.where(d["table"] >= 0, move[d["table"]], -1).astype(np.int32))
    q = dev_bf16(d["q"])
    at = torch.from_numpy(move).cuda()
    if fp8:
        cache = (torch.zeros(pool, 64, 576, dtype=torch.uint8, device="cuda"),
                 torch.zeros(pool, 64, dtype=torch.int8, device="cuda"))
        cache[0][at] = torch.from_numpy(d["codes"]).cuda()
        cache[1][at] = torch.from_numpy(d["exps"]).cuda()
        call = mla.decode_attention_shared_fp8
    else:
        cache = (torch.zeros(pool, 64, 576, dtype=torch.bfloat16, device="cuda"),)
        cache[0][at] = dev_bf16(d["bits"])
        call = mla.decode_attention_shared
    out, lse, ws = call(q[..., :512].contiguous(), q[..., 512:].contiguous(), *cache,
                        dev_i32(big["table"]), dev_i32(d["lens"]), dev_i32(d["groups"]),
                        dev_i32(d["prefix"]), max(d["lens"]), d["scale"])
    check(d, out, lse, mla.check_device_status(ws))


def test_sequences_before_the_first_group(mla):
    d = shared_case(17, 16, 2, [(0, [5, 300, 0]), (700, [701 + 31 * i for i in range(9)]), (0, [77])])
    d["groups"], d["prefix"] = np.array([3, 12], np.int32), np.array([700], np.int32)
    check(d, *run(mla, d))
    # and groups without sequences
    d["groups"] = np.array([3, 3, 12, 12, 12], np.int32)
    d["prefix"] = np.array([64, 700, 5, 10 ** 9], np.int32)
    check(d, *run(mla, d))


def test_two_streams_at_once(mla):
    """Calls that overlap on the GPU, each with its own workspace."""
    ds = [shared_case(18 + k, 32, 1, [(3000, [3001 + 40 * i + k for i in range(20)])]) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in ds]
    args, outs = [], []
    for d in ds:
        q = dev_bf16(d["q"])
        args.append((q[..., :512].contiguous(), q[..., 512:].contiguous(), dev_bf16(d["bits"]),
                     dev_i32(d["table"]), dev_i32(d["lens"]), dev_i32(d["groups"]), dev_i32(d["prefix"]),
                     max(d["lens"]), d["scale"]))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [mla.decode_attention_shared(*a, stream=st) for a, st in zip(args, streams)]
    torch.cuda.synchronize()
    for d, (out, lse, ws) in zip(ds, outs):
        check(d, out, lse, mla.check_device_status(ws))
