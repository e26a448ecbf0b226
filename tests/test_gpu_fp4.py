"""The 4-bit latent cache: quantised as it is written, and rows of every cache format read back,
against the format's definition (tests/fp4_ref.py) and the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from mla_latent_kv_13_gb300 import synth
from tests import fp4_ref as F
from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_f64_from_bf16

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def pages(rng, lens, spare=2):
    blocks = max(1, max(-(-n // 64) for n in lens))
    pool = sum(-(-n // 64) for n in lens) + spare
    table = np.full((len(lens), blocks), -1, np.int32)
    order, at = rng.permutation(pool), 0
    for b, n in enumerate(lens):
        k = -(-n // 64)
        table[b, :k] = order[at:at + k]
        at += k
    return table, pool


def inputs(seed, counts, lens, q_lora, pad=0, spread=1.0):
    rng = np.random.default_rng(seed)
    tokens = sum(counts) + pad
    x = rng.standard_normal((tokens, q_lora + 576)) * np.exp(spread * rng.standard_normal((tokens, 1)))
    x[:, q_lora:q_lora + 512] *= np.exp(1.5 * rng.standard_normal((tokens, 512)))
    table, pool = pages(rng, lens)
    return dict(x=R.bf16_bits(x.astype(np.float32)), q_lora=q_lora, counts=counts, lens=lens,
                w_q=R.bf16_bits(1 + 0.3 * rng.standard_normal(q_lora).astype(np.float32)),
                w_kv=R.bf16_bits(1 + 0.3 * rng.standard_normal(512).astype(np.float32)),
                table=table, pool=pool,
                starts=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def to_bf16(x):
    """fp64 to the nearest of 8 significant bits, ties to even (values inside bf16's normal range)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def reference(d, plan, eps=EPS):
    """c_q, the latent rows rounded to bf16, the rotated keys, and the rows' places."""
    f = synth.bf16_bits_to_f64
    x, ql, n = f(d["x"]), d["q_lora"], int(d["starts"][-1])

    def rms(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * f(w)

    c_q = rms(x[:n, :ql], d["w_q"]) if ql else np.zeros((n, 0))
    latent = to_bf16(rms(x[:n, ql:ql + 512], d["w_kv"]))
    keys, place = np.zeros((n, 64)), np.zeros((n, 2), int)
    freq = np.array(plan.freq[:32])
    r = x[:, ql + 512:]
    a, b = (r[:, :32], r[:, 32:]) if plan.layout else (r[:, 0::2], r[:, 1::2])
    for s, (c, length) in enumerate(zip(d["counts"], d["lens"])):
        for i in range(c):
            t, p = int(d["starts"][s]) + i, length - c + i
            z = plan.magnitude * (a[t] + 1j * b[t]) * np.exp(1j * p * freq)
            if plan.layout:
                keys[t] = np.concatenate([z.real, z.imag])
            else:
                keys[t, 0::2], keys[t, 1::2] = z.real, z.imag
            place[t] = (d["table"][s, p // 64], p % 64)
    size = plan.magnitude * np.hypot(a[:n], b[:n])
    size = np.concatenate([size, size], 1) if plan.layout else np.repeat(size, 2, 1)
    # half a step, and fp32 arithmetic with an angle good to 2^-22 of a turn
    ktol = 2.0 ** -8 * np.abs(keys) + 2.0 ** -20 * size + 1e-38
    return c_q, latent, keys, ktol, place


def cache4(pool, fill=0x5A):
    c = torch.full((pool, 64, 256), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((pool, 64, 32), fill, dtype=torch.uint8, device="cuda")
    e = torch.full((pool, 64), fill, dtype=torch.int8, device="cuda")
    k = torch.full((pool, 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    return c, s, e, k


def append(mla, d, cache, plan, eps=EPS, **kw):
    c_q, ws = mla.norm_rope_append_fp4(dev_bf16(d["x"]), dev_bf16(d["w_q"]), dev_bf16(d["w_kv"]),
                                       dev_i32(d["starts"]), dev_i32(d["lens"]), dev_i32(d["table"]),
                                       *cache, plan, eps, **kw)
    return c_q, mla.check_device_status(ws)


def check_append(mla, d, plan, eps=EPS):
    cache = cache4(d["pool"])
    c_q, status = append(mla, d, cache, plan, eps)
    assert status == 0
    wq, latent, keys, ktol, place = reference(d, plan, eps)
    n = len(latent)
    got = host_f64_from_bf16(c_q)[:n]
    assert np.all(np.abs(got - wq) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(wq))
    assert not c_q[n:].any()  # a padded batch's tokens
    codes, scales, exps = F.quantize(latent)
    pg, sl = place[:, 0], place[:, 1]
    host = [t.cpu().numpy() for t in cache[:3]]
    assert np.array_equal(host[2][pg, sl].astype(int), exps)
    assert np.array_equal(host[1][pg, sl].astype(int), scales)
    got = F.unpack(host[0])[pg, sl]
    got[got == 8] = 0  # a zero's sign is not specified
    assert np.array_equal(got, codes)
    k = host_f64_from_bf16(cache[3])[pg, sl]
    assert np.all(np.abs(k - keys) <= ktol)
    # nothing else was written
    seen = np.zeros((d["pool"], 64), bool)
    seen[pg, sl] = True
    assert (host[0][~seen] == 0x5A).all() and (host[1][~seen] == 0x5A).all()
    assert (host[2][~seen] == 0x5A).all() and (cache[3].float().cpu().numpy()[~seen] == 3.0).all()
    return cache, place, F.values(codes, scales, exps), k


CASES = {
    "decode": ([1] * 9, [1, 64, 65, 7, 700, 128, 3, 2, 1000], 1536, 0),
    "prompts": ([70, 1, 0, 130], [70, 33, 5, 200], 64, 3),
    "no queries": ([5, 9], [64, 9], 0, 0),
    "one": ([1], [1], 8, 1),
}


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("name", list(CASES))
def test_append_fp4(mla, name, layout):
    counts, lens, ql, pad = CASES[name]
    d = inputs(1, counts, lens, ql, pad)
    check_append(mla, d, mla.rope_plan(scaling="yarn", factor=40.0, original=4096, layout=layout))


@pytest.mark.parametrize("spread", [0.0, 0.5, 3.0, 8.0])
def test_every_scale(mla, spread):
    """Rows whose groups differ by many powers of two: scales down to the least and to zero."""
    rng = np.random.default_rng(3)
    n = 300
    x = rng.standard_normal((n, 32, 16)) * np.exp2(spread * rng.standard_normal((n, 32, 1)))
    d = inputs(2, [n], [n], 0)
    d["x"][:, :512] = R.bf16_bits(x.reshape(n, 512).astype(np.float32))
    d["x"][5, :512] = 0  # a row of zeros
    d["x"][6, 16:512] = 0
    check_append(mla, d, mla.rope_plan())


def test_ties(mla):
    """Rows of few significant bits, where codes, scales and roundings lie on borders: rows of equal
    magnitudes have a norm of one over it, so what is stored is the weight."""
    rng = np.random.default_rng(4)
    n = 64
    d = inputs(3, [n], [n], 0)
    d["x"][:, :512] = R.bf16_bits(np.where(rng.random((n, 512)) < 0.5, -4096.0, 4096.0).astype(np.float32))
    for k in range(8):
        w = rng.integers(0, 97, 512) / 8.0 * 2.0 ** k
        w[::16] = 6.0 * 2.0 ** k * rng.choice([1, 1.0625, 1.125, 1.1875, 1.9375], 32)
        d["w_kv"] = R.bf16_bits(w.astype(np.float32))
        check_append(mla, d, mla.rope_plan())


def test_largest(mla):
    """Values up to bf16's largest: they stay finite."""
    d = inputs(4, [3], [3], 0)
    d["x"][:, :512] = R.bf16_bits(np.full((3, 512), 4096.0, np.float32))
    rng = np.random.default_rng(5)
    w = rng.integers(128, 256, 512) * 2.0 ** 120
    w[5] = 255 * 2.0 ** 120
    d["w_kv"] = R.bf16_bits(w.astype(np.float32))
    cache, _, value, _ = check_append(mla, d, mla.rope_plan())
    out, _ = mla.read_kv_fp4(*cache, dev_i32(d["table"]), None, dev_i32([0, 3]), rows=3)
    assert np.array_equal(host_f64_from_bf16(out)[:, :512], value) and np.isfinite(value).all()


@pytest.mark.parametrize("x_power,w_power", [(-100, 100), (-60, -50), (100, -100), (60, 60), (-120, 0),
                                             (120, 5), (-20, -95)])
def test_products_out_of_range(mla, x_power, w_power):
    """Without an epsilon the size of x does not matter, also where its products with the weights or
    its squares are outside fp32's range."""
    d = inputs(6, [20], [20], 0, spread=0.1)
    x = synth.bf16_bits_to_f64(d["x"])[:, :512]
    d["x"][:, :512] = R.bf16_bits((x * 2.0 ** x_power).astype(np.float32))
    w = synth.bf16_bits_to_f64(d["w_kv"])
    d["w_kv"] = R.bf16_bits((w * 2.0 ** w_power).astype(np.float32))
    check_append(mla, d, mla.rope_plan(), eps=0.0)


@pytest.mark.parametrize("power", [-130, -100, -60, 60, 100, 125])
def test_magnitudes(mla, power):
    """Weights and inputs of every magnitude (the norm takes the inputs' out): e from its lowest."""
    d = inputs(5, [40], [40], 0)
    x = synth.bf16_bits_to_f64(d["x"])
    if power > -100:
        x = x[:, :512] / np.abs(x[:, :512]).max() * 2.0 ** min(power, 60)
        d["x"][:, :512] = R.bf16_bits(x.astype(np.float32))
    w = synth.bf16_bits_to_f64(d["w_kv"]) * 2.0 ** min(power, 118)
    d["w_kv"] = R.bf16_bits(w.astype(np.float32))
    cache = cache4(d["pool"])
    _, status = append(mla, d, cache, mla.rope_plan())
    assert status == 0
    f = synth.bf16_bits_to_f64
    v = f(d["x"])[:, :512]
    exact = v / np.sqrt((v * v).mean(-1, keepdims=True) + EPS) * f(d["w_kv"])
    out, ws = mla.read_kv_fp4(*cache, dev_i32(d["table"]), None, dev_i32([0, 40]), rows=40)
    assert mla.check_device_status(ws) == 0
    got = host_f64_from_bf16(out)[:, :512]
    assert np.isfinite(got).all()
    # at worst half the gap of the levels 4 and 6, one scale, which is at most 17/16 of a sixth of the
    # largest of the 16; where the scale is subnormal, 6 of its steps of 2^-9
    g = np.abs(exact).reshape(40, 32, 16).max(2)
    floor = 6 * 2.0 ** -9 * 2.0 ** np.maximum(np.ceil(np.log2(np.abs(exact).max(1) / 2688)), -120)
    tol = np.repeat(np.maximum(g / 5, floor[:, None]), 16, 1)
    assert (np.abs(got - exact) <= tol).all()


def test_not_finite(mla):
    """A NaN in a row makes its latents NaN (the norm spreads it); the other rows and the keys are as
    they were. The key of a row is kept apart from its latents."""
    d = inputs(6, [8], [8], 0)
    clean, _, _, _ = check_append(mla, d, mla.rope_plan())
    d["x"][3, 17] = 0x7FC0
    d["x"][5, 40] = 0x7F80
    d["x"][6, 512] = 0x7FC0
    cache = cache4(d["pool"])
    _, status = append(mla, d, cache, mla.rope_plan())
    assert status == 0
    out, _ = mla.read_kv_fp4(*cache, dev_i32(d["table"]), None, dev_i32([0, 8]), rows=8)
    want, _ = mla.read_kv_fp4(*clean, dev_i32(d["table"]), None, dev_i32([0, 8]), rows=8)
    assert torch.isnan(out[3, :512]).all() and torch.isfinite(out[3, 512:]).all()
    assert torch.isnan(out[5, 32:48]).all()
    for row in (0, 1, 2, 4, 7):
        assert torch.equal(out[row], want[row])
    assert torch.equal(out[6, :512], want[6, :512]) and torch.isnan(out[6, 512:514]).all()
    assert torch.equal(out[6, 514:], want[6, 514:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_append_scaled(mla, fp8, layout):
    """The bf16 and FP8 appends with a plan: the latents those of the call without, the keys turned as
    the plan says; with theta's own frequencies the same bits."""
    d = inputs(7, [30, 1, 5], [90, 64, 5], 128)
    n = 36
    args = (dev_bf16(d["x"]), dev_bf16(d["w_q"]), dev_bf16(d["w_kv"]), dev_i32(d["starts"]),
            dev_i32(d["lens"]), dev_i32(d["table"]))

    def new():
        if fp8:
            return (torch.zeros(d["pool"], 64, 576, dtype=torch.uint8, device="cuda"),
                    torch.zeros(d["pool"], 64, dtype=torch.int8, device="cuda"))
        return (torch.zeros(d["pool"], 64, 576, dtype=torch.bfloat16, device="cuda"),)

    plain, same, other = new(), new(), new()
    (mla.norm_rope_append_fp8 if fp8 else mla.norm_rope_append)(*args, *plain, 10000.0, EPS)
    call = mla.norm_rope_append_scaled_fp8 if fp8 else mla.norm_rope_append_scaled
    c_q, ws = call(*args, *same, mla.rope_plan(), EPS)
    assert mla.check_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(plain, same))
    plan = mla.rope_plan(scaling="bands", factor=8.0, original=100, fast=4.0, layout=layout, magnitude=1.25)
    call(*args, *other, plan, EPS)
    _, _, keys, ktol, place = reference(d, plan)
    pg, sl = place[:, 0], place[:, 1]
    if fp8:
        got = R.fp8_values(*(t.cpu().numpy() for t in other))[pg, sl]
        # a code's half step, 2^-4 of the value, or of the least normal, 2^-7 of the scale
        ktol = ktol + 2.0 ** -4 * np.abs(keys) + 2.0 ** -10 * 2.0 ** other[1].cpu().numpy()[pg, sl][:, None].astype(float)
    else:
        got = host_f64_from_bf16(other[0])[pg, sl]
        assert torch.equal(other[0][..., :512], plain[0][..., :512])
    assert np.all(np.abs(got[:, 512:] - keys) <= ktol)


def spans(case):
    rng = np.random.default_rng(case["seed"])
    first, n = case["first"], case["n"]
    lens = [f + k for f, k in zip(first, n)]
    table, pool = pages(rng, lens)
    starts = np.concatenate([[case.get("at", 0)], case.get("at", 0) + np.cumsum(n)]).astype(np.int32)
    return rng, table, pool, starts


READS = {
    "one row": dict(first=[0], n=[1]),
    "ragged": dict(first=[0, 64, 63, 5, 200, 0], n=[64, 65, 2, 0, 300, 1]),
    "many short": dict(first=list(range(100)), n=[k % 4 for k in range(100)]),
    "as many as may be": dict(first=[k % 70 for k in range(4096)], n=[(k * 7) % 3 for k in range(4096)]),
    "long": dict(first=[7], n=[5000]),
    "padded": dict(first=[0, 10], n=[70, 90], at=13, pad=9),
}


def filled(rng, pool, kind):
    """A cache of random contents (every code, no NaN) and the values that it stands for."""
    if kind == "bf16":
        bits = R.bf16_bits(rng.standard_normal((pool, 64, 576)).astype(np.float32))
        return (dev_bf16(bits),), synth.bf16_bits_to_f64(bits)
    exps = rng.integers(-20, 8, (pool, 64)).astype(np.int8)
    if kind == "fp8":
        codes = rng.integers(0, 256, (pool, 64, 576)).astype(np.uint8)
        codes[(codes & 127) == 127] = 5
        return (torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda()), R.fp8_values(codes, exps)
    codes = rng.integers(0, 16, (pool * 64, 512))
    scales = rng.integers(0, 127, (pool * 64, 32)).astype(np.uint8)
    keys = R.bf16_bits(rng.standard_normal((pool, 64, 64)).astype(np.float32))
    v = F.values(codes, scales.astype(int), exps.reshape(-1)).reshape(pool, 64, 512)
    cache = (torch.from_numpy(F.pack(codes).reshape(pool, 64, 256)).cuda(),
             torch.from_numpy(scales.reshape(pool, 64, 32)).cuda(), torch.from_numpy(exps).cuda(),
             dev_bf16(keys))
    return cache, np.concatenate([v, synth.bf16_bits_to_f64(keys)], 2)


def read(mla, kind):
    return dict(bf16=mla.read_kv, fp8=mla.read_kv_fp8, fp4=mla.read_kv_fp4)[kind]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("name", list(READS))
def test_read(mla, name, kind):
    case = dict(READS[name], seed=8)
    rng, table, pool, starts = spans(case)
    cache, value = filled(rng, pool, kind)
    rows = int(starts[-1]) + case.get("pad", 0)
    out = torch.full((rows, 576), 9.0, dtype=torch.bfloat16, device="cuda")
    got, ws = read(mla, kind)(*cache, dev_i32(table), dev_i32(case["first"]), dev_i32(starts), out=out)
    assert got is out and mla.check_device_status(ws) == 0
    want = np.full((rows, 576), 9.0)
    for b, (f, n) in enumerate(zip(case["first"], case["n"])):
        p = np.arange(f, f + n)
        want[starts[b]:starts[b] + n] = value[table[b, p // 64], p % 64]
    assert np.array_equal(host_f64_from_bf16(out), want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_read_bad_places(mla, kind):
    """Bad page ids, positions before the first and behind the last page: rows of zeros, recorded."""
    rng = np.random.default_rng(9)
    cache, value = filled(rng, 4, kind)
    table = np.array([[0, 4, 2], [-1, 1, 2 ** 31 - 1]], np.int32)
    first, n = [-2, 100], [140, 100]
    starts = np.array([0, 140, 240], np.int32)
    out, ws = read(mla, kind)(*cache, dev_i32(table), dev_i32(first), dev_i32(starts), rows=240)
    assert mla.check_device_status(ws) == 4
    got = host_f64_from_bf16(out)
    for b in range(2):
        for i in range(n[b]):
            p = first[b] + i
            ok = 0 <= p < 192 and 0 <= table[b, p // 64] < 4
            assert np.array_equal(got[starts[b] + i], value[table[b, p // 64], p % 64] if ok else np.zeros(576))
    # ranges that do not ascend within [0, rows] are recorded
    for bad in ([0, 9, 5], [-1, 3, 9], [0, 3, 241], [2 ** 31 - 1, -2 ** 31, 7]):
        _, ws = read(mla, kind)(*cache, dev_i32(table), dev_i32(first), dev_i32(np.array(bad)), out=out)
        assert mla.check_device_status(ws) == 4


def test_read_every_code(mla):
    """Each of the 16 codes under each scale and the ends of the exponents' range, NaN scales too."""
    scales = np.repeat(np.arange(128, dtype=np.uint8)[:, None], 32, 1)
    codes = np.tile(np.arange(16), (128, 32))
    keys = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    for e in (-120, -7, 0, 100):
        exps = np.full(128, e)
        want = F.values(codes, scales.astype(int), exps)
        cache = (torch.from_numpy(F.pack(codes).reshape(2, 64, 256)).cuda(),
                 torch.from_numpy(scales.reshape(2, 64, 32)).cuda(),
                 torch.full((2, 64), e, dtype=torch.int8, device="cuda"), keys)
        out, ws = mla.read_kv_fp4(*cache, dev_i32([[0, 1]]), None, dev_i32([0, 128]), rows=128)
        assert mla.check_device_status(ws) == 0
        got = host_f64_from_bf16(out)[:, :512]
        assert np.array_equal(got, want, equal_nan=True)


def test_append_bad_places(mla):
    d = inputs(10, [3, 2], [2, 70], 0)
    d["table"][1, 1] = 99
    cache = cache4(d["pool"])
    _, status = append(mla, d, cache, mla.rope_plan())
    assert status == 4  # a token before the first row, and a page out of the pool
    written = (cache[2] != 0x5A).sum()
    assert int(written) == 2  # the two tokens of the first sequence that have rows


def test_pools_fork_and_compact(mla):
    """The four pools of a 4-bit cache go through the pages' calls."""
    rng = np.random.default_rng(11)
    cache, value = filled(rng, 12, "fp4")
    refs = torch.zeros(12, dtype=torch.int32, device="cuda")
    table = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    table[0, :2] = dev_i32([9, 7])
    lens[0] = 100
    refs[9] = refs[7] = 1
    pools = [t[None] for t in cache]
    ws = mla.pages_fork(refs, table, lens, dev_i32([0, 0]), dev_i32([2, 3]), pools)
    assert mla.check_device_status(ws) == 0
    _, _, live, ws = mla.pages_compact(refs, table, lens, pools, workspace=ws)
    assert mla.check_device_status(ws) == 0 and int(live) == 4
    want = np.concatenate([value[9], value[7][:36]])
    out, ws = mla.read_kv_fp4(*cache, table, None, dev_i32([0, 100, 100, 200, 300]), rows=300)
    assert mla.check_device_status(ws) == 0
    got = host_f64_from_bf16(out)
    for k in range(3):
        assert np.array_equal(got[100 * k:100 * k + 100], want)


def test_graph_and_stream(mla):
    """A captured write and read serve other tokens; a stream of its own."""
    plan = mla.rope_plan(scaling="yarn", factor=40.0, original=4096)
    a, b = inputs(12, [40, 1], [50, 70], 64), inputs(13, [20, 21], [70, 64], 64)
    b["table"], b["pool"] = a["table"], a["pool"]
    b["lens"] = [50, 70]
    b["table"] = a["table"]
    held = [dev_bf16(a["x"]), dev_bf16(a["w_q"]), dev_bf16(a["w_kv"]), dev_i32(a["starts"]),
            dev_i32(a["lens"]), dev_i32(a["table"])]
    cache = cache4(a["pool"])
    c_q = torch.zeros(41, 64, dtype=torch.bfloat16, device="cuda")
    first, starts = dev_i32([0, 0]), dev_i32([0, 50, 120])
    out = torch.zeros(120, 576, dtype=torch.bfloat16, device="cuda")
    ws = mla.alloc_workspace(0)

    def step(stream=None):
        mla.norm_rope_append_fp4(*held, *cache, plan, EPS, c_q=c_q, workspace=ws, stream=stream)
        mla.read_kv_fp4(*cache, held[5], first, starts, out=out, workspace=ws, stream=stream)

    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(st)
    st.synchronize()
    assert mla.check_device_status(ws) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for d in (b, a):
        for to, k in zip(held, ("x", "w_q", "w_kv")):
            to.copy_(dev_bf16(d[k]))
        held[3].copy_(dev_i32(d["starts"])), held[4].copy_(dev_i32(d["lens"]))
        g.replay()
        torch.cuda.synchronize()
        assert mla.check_device_status(ws) == 0
        _, latent, _, _, place = reference(d, plan)
        value = F.values(*F.quantize(latent))
        got, at = host_f64_from_bf16(out)[:, :512], 0
        for s, (c, n) in enumerate(zip(d["counts"], d["lens"])):
            new = got[starts[s].item() + n - c:starts[s].item() + n]
            assert np.array_equal(new, value[at:at + c])
            at += c


def test_refused(mla):
    d = inputs(14, [2], [2], 0)
    cache = cache4(d["pool"])
    with pytest.raises(mla.MLAError):  # a key is 64 values
        append(mla, d, cache, mla.rope_plan(32))
    with pytest.raises(ValueError):
        append(mla, d, (cache[0][..., :128].contiguous(), *cache[1:]), mla.rope_plan())
    with pytest.raises(TypeError):
        append(mla, d, (*cache[:3], cache[3].float()), mla.rope_plan())
    with pytest.raises(ValueError):
        mla.read_kv_fp4(*cache, dev_i32(d["table"]), None, dev_i32([0, 1, 2]), rows=2)
    with pytest.raises(ValueError):
        mla.read_kv(torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda"), dev_i32(d["table"]),
                    None, dev_i32([0, 1]))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_far_pages(mla, kind):
    """Pages whose bytes and values lie behind 2^31 and 2^32 of the cache's start."""
    rng = np.random.default_rng(16)
    small, value = filled(rng, 3, kind)
    pool = dict(bf16=70000, fp8=130000, fp4=290000)[kind]
    ids = [pool - 1, 5, pool - 2]
    cache = []
    for t in small:
        big = torch.zeros((pool, *t.shape[1:]), dtype=t.dtype, device="cuda")
        big[ids] = t
        cache.append(big)
    out, ws = read(mla, kind)(*cache, dev_i32([ids]), None, dev_i32([0, 192]), rows=192)
    assert mla.check_device_status(ws) == 0
    assert np.array_equal(host_f64_from_bf16(out), value.reshape(192, 576))
    if kind != "fp4":
        return
    d = inputs(17, [70], [70], 0)
    d["table"] = np.array([[pool - 3, pool - 1]], np.int32)
    _, status = append(mla, d, cache, mla.rope_plan())
    assert status == 0
    _, latent, _, _, place = reference(d, mla.rope_plan())
    out, ws = mla.read_kv_fp4(*cache, dev_i32(d["table"]), None, dev_i32([0, 70]), rows=70)
    assert np.array_equal(host_f64_from_bf16(out)[:, :512], F.values(*F.quantize(latent)))
