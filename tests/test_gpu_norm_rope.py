"""The latent norms with the rotation and the cache write, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from mla_latent_kv_13_gb300 import synth
from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_bits, host_f64_from_bf16

pytestmark = pytest.mark.gpu

EPS, THETA = 1e-6, 10000.0


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def inputs(seed, counts, lens, q_lora, pad=0, spread=1.0):
    rng = np.random.default_rng(seed)
    tokens = sum(counts) + pad
    x = rng.standard_normal((tokens, q_lora + 576)) * np.exp(
        spread * rng.standard_normal((tokens, 1)))
    blocks = max(1, max(-(-n // 64) for n in lens))
    pool = sum(-(-n // 64) for n in lens) + 2
    table = np.full((len(lens), blocks), -1, np.int32)
    order, at = rng.permutation(pool), 0
    for b, n in enumerate(lens):
        k = -(-n // 64)
        table[b, :k] = order[at:at + k]
        at += k
    return dict(x=R.bf16_bits(x.astype(np.float32)), q_lora=q_lora, counts=counts, lens=lens,
                w_q=R.bf16_bits(1 + 0.3 * rng.standard_normal(q_lora).astype(np.float32)),
                w_kv=R.bf16_bits(1 + 0.3 * rng.standard_normal(512).astype(np.float32)),
                table=table, pool=pool,
                starts=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def reference(d):
    """c_q and the key rows with their places, in 64 bits."""
    f = synth.bf16_bits_to_f64
    x, ql = f(d["x"]), d["q_lora"]

    def rms(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + EPS) * f(w)

    n = int(d["starts"][-1])
    c_q = rms(x[:n, :ql], d["w_q"]) if ql else np.zeros((n, 0))
    rows = np.zeros((n, 576))
    rows[:, :512] = rms(x[:n, ql:ql + 512], d["w_kv"])
    place = np.zeros((n, 2), int)
    freq = THETA ** (-2.0 * np.arange(32) / 64)
    for b, (c, length) in enumerate(zip(d["counts"], d["lens"])):
        for i in range(c):
            t, p = int(d["starts"][b]) + i, length - c + i
            z = (x[t, ql + 512::2] + 1j * x[t, ql + 513::2]) * np.exp(1j * p * freq)
            rows[t, 512::2], rows[t, 513::2] = z.real, z.imag
            place[t] = (d["table"][b, p // 64], p % 64)
    # before the rounding: fp32 sums and factors (under 2^-20 relative together); a rotated pair
    # errs by that much of its length, with an angle good to 2^-22 of a turn
    slack = 2.0 ** -20 * np.abs(rows)
    pair = np.hypot(rows[:, 512::2], rows[:, 513::2])
    slack[:, 512:] = 2.0 ** -20 * np.repeat(pair, 2, 1)
    return c_q, rows, place, slack


def run(mla, d, cache, **kw):
    call = mla.norm_rope_append if len(cache) == 1 else mla.norm_rope_append_fp8
    c_q, ws = call(dev_bf16(d["x"]), dev_bf16(d["w_q"]), dev_bf16(d["w_kv"]),
                   dev_i32(d["starts"]), dev_i32(d["lens"]), dev_i32(d["table"]), *cache, THETA,
                   EPS, **kw)
    return c_q, mla.check_device_status(ws)


CASES = {
    "decode": ([1] * 9, [1, 64, 65, 7, 700, 128, 3, 2, 1000], 1536),
    "mixed": ([5, 0, 1, 70, 64], [5, 3, 900, 200, 64], 128),
    "no queries": ([3, 1], [100, 1], 0),
    "narrow": ([2, 2], [70, 2], 8),
    "wide": ([3], [65], 4000),
    "single": ([1], [1], 1536),
}


@pytest.mark.parametrize("name", list(CASES))
def test_bf16(mla, name):
    counts, lens, ql = CASES[name]
    d = inputs(1, counts, lens, ql)
    cache = torch.full((d["pool"], 64, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    c_q, st = run(mla, d, (cache,))
    assert st == 0
    ref, rows, place, slack = reference(d)
    half = R.HALF_STEP_BF16
    R.assert_within(host_f64_from_bf16(c_q), ref, (half + 2.0 ** -20) * np.abs(ref) + 1e-30, "c_q")
    got = host_f64_from_bf16(cache)
    R.assert_within(got[place[:, 0], place[:, 1]], rows,
                    half * (np.abs(rows) + slack) + slack + 1e-30, "rows")
    got[place[:, 0], place[:, 1]] = 3.0
    assert (got == 3.0).all()  # no other row was touched


@pytest.mark.parametrize("name", list(CASES))
def test_fp8(mla, name):
    counts, lens, ql = CASES[name]
    d = inputs(2, counts, lens, ql, spread=3.0)
    codes = torch.full((d["pool"], 64, 576), 9, dtype=torch.uint8, device="cuda")
    exps = torch.full((d["pool"], 64), 5, dtype=torch.int8, device="cuda")
    c_q, st = run(mla, d, (codes, exps))
    assert st == 0
    ref, rows, place, slack = reference(d)
    R.assert_within(host_f64_from_bf16(c_q), ref,
                    (R.HALF_STEP_BF16 + 2.0 ** -20) * np.abs(ref) + 1e-30, "c_q")
    k, e = codes.cpu().numpy(), exps.cpu().numpy()
    at = (place[:, 0], place[:, 1])
    # the smallest exponent with max |row| 2^-e <= 448 (random rows: never within 2^-20 of it)
    top = np.abs(rows).max(1)
    want = np.ceil(np.log2(top / 448)).astype(int)
    assert (np.abs(np.log2(top / 448) - np.round(np.log2(top / 448))) > 1e-5).all()
    assert np.array_equal(e[at], np.maximum(want, -126))
    step = 2.0 ** e[at].astype(float)[:, None]
    got = R.fp8_values(k[at], e[at])
    # e4m3: half a step of 3 mantissa bits, or of the subnormals
    R.assert_within(got, rows, 2.0 ** -4 * np.abs(rows) + 2.0 ** -10 * step + 2 * slack, "rows")
    untouched = np.ones(e.shape, bool)
    untouched[at] = False
    assert (k[untouched] == 9).all() and (e[untouched] == 5).all()


def test_padded_batch_and_strided_rows(mla):
    d = inputs(3, [4, 30], [90, 40], 64, pad=5)
    wide = torch.zeros((39, 64 + 576 + 24), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:648] = dev_bf16(d["x"])
    cache = torch.zeros((d["pool"], 64, 576), dtype=torch.bfloat16, device="cuda")
    c_q = torch.full((39, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, ws = mla.norm_rope_append(wide[:, 8:648], dev_bf16(d["w_q"]), dev_bf16(d["w_kv"]),
                                 dev_i32(d["starts"]), dev_i32(d["lens"]), dev_i32(d["table"]),
                                 cache, THETA, EPS, c_q=c_q)
    assert mla.check_device_status(ws) == 0
    assert (c_q[34:] == 7).all()
    plain = torch.zeros_like(cache)
    d["x"] = d["x"][:34]
    c2, st = run(mla, d, (plain,))
    assert st == 0 and torch.equal(c2, c_q[:34])
    assert torch.equal(plain.view(torch.int16), cache.view(torch.int16))


def test_zero_row_and_far_positions(mla):
    d = inputs(4, [2, 1], [2, 1], 16)
    d["x"][0] = 0
    d["lens"] = [2, 3_000_001]
    d["table"] = np.full((2, 3_000_001 // 64 + 1), -1, np.int32)
    d["table"][0, 0], d["table"][1, -1] = 1, 0
    cache = torch.zeros((d["pool"], 64, 576), dtype=torch.bfloat16, device="cuda")
    c_q, st = run(mla, d, (cache,))
    assert st == 0
    ref, rows, place, slack = reference(d)
    got = host_f64_from_bf16(cache)[place[:, 0], place[:, 1]]
    # the reference's own angles err here: 3e6 radians in fp64 are good to 1e-9
    R.assert_within(got, rows, R.HALF_STEP_BF16 * (np.abs(rows) + slack) + slack + 1e-8, "rows")
    assert (c_q[0] == 0).all()


def test_bad_places_are_recorded_and_only_their_rows_dropped(mla):
    d = inputs(5, [3, 2, 1], [2, 100, 30], 8)  # sequence 0 brings more tokens than it has rows
    d["table"][2, 0] = d["pool"]
    cache = torch.full((d["pool"], 64, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    c_q, st = run(mla, d, (cache,))
    assert st == 4
    got = host_f64_from_bf16(cache)
    touched = (got != 3.0).any(-1)
    want = np.zeros_like(touched)
    for b, p in ((0, 0), (0, 1), (1, 98), (1, 99)):
        want[d["table"][b, p // 64], p % 64] = True
    assert np.array_equal(touched, want)
    assert (c_q != 0).any(-1).all()


def test_many_sequences(mla):
    counts = [k % 3 for k in range(1500)]
    d = inputs(6, counts, [c + 5 for c in counts], 64)
    cache = torch.zeros((d["pool"], 64, 576), dtype=torch.bfloat16, device="cuda")
    c_q, st = run(mla, d, (cache,))
    assert st == 0
    ref, rows, place, slack = reference(d)
    R.assert_within(host_f64_from_bf16(cache)[place[:, 0], place[:, 1]], rows,
                    R.HALF_STEP_BF16 * (np.abs(rows) + slack) + slack + 1e-30, "rows")


@pytest.mark.parametrize("B", [1, 31, 32, 33, 64, 65, 127, 128, 129, 300, 4096])
def test_every_batch_size_finds_its_sequences(mla, B):
    """Sequences of no, one and several tokens, in batches around the widths of the search: each
    token's row lands at its own position of its own sequence, and padding's nowhere."""
    rng = np.random.default_rng(B)
    counts = rng.choice([0, 1, 1, 2, 5], B)
    counts[rng.integers(B)] = 3
    starts = np.r_[2, 2 + np.cumsum(counts)].astype(np.int32)
    T = int(starts[-1]) + 3
    lens = (counts + rng.integers(0, 60, B)).astype(np.int32)
    x = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1 + torch.arange(T, device="cuda") % 200 / 256  # (normed to the same; the sign tells)
    x[:, 1] = 1
    sign = torch.where(torch.arange(T, device="cuda") % 3 == 0, -1.0, 1.0)
    x[:, 0] *= sign.to(torch.bfloat16)
    cache = torch.full((B, 64, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    _, ws = mla.norm_rope_append(x, None, w, dev_i32(starts), dev_i32(lens), table, cache)
    assert mla.check_device_status(ws) == 0
    got = cache[:, :, :2].float().cpu().numpy()
    want = np.full((B, 64, 2), 7.0)
    xs = x[:, :2].double().cpu().numpy()
    for b in range(B):
        for i in range(counts[b]):
            v = xs[starts[b] + i]
            want[b, lens[b] - counts[b] + i] = v / np.sqrt((v * v).sum() / 512 + 1e-6)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1e-6)
