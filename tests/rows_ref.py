"""Plain 64-bit forms of the ragged serving operators, and the inputs and bounds of their tests."""
import numpy as np

from mla_latent_kv_13_gb300 import synth

PAGE, D_C, D_R, D = 64, 512, 64, 576
SCALE = 1.0 / np.sqrt(192.0)
HALF_STEP_BF16 = 2.0 ** -8  # half a step of bf16, relative to the value


def bf16_bits(x):
    """Nearest-even bf16 bit patterns of finite fp32 values."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def visible(length, count, i, window, sinks):
    """The rows that token i of a sequence's `count` new ones sees."""
    p = length - count + i
    j = np.arange(max(p + 1, 0))
    if window:
        j = j[(j > p - window) | (j < sinks)]
    return j


def attention_case(seed, heads, counts, lens, window=0, sinks=0, spare=3, pad=0, fp8=False,
                   scale=SCALE, size=0.6):
    """Inputs of a ragged batch: pages in shuffled order, pages that no token sees not there
    (table entry -1), and NaN in every cached row that no token sees."""
    rng = np.random.default_rng(seed)
    B, tokens = len(counts), int(sum(counts))
    blocks = max(1, max((n + PAGE - 1) // PAGE for n in lens))
    seen = [np.unique(np.concatenate([visible(n, c, i, window, sinks) for i in range(c)] or
                                     [np.zeros(0, int)])).astype(int) for c, n in zip(counts, lens)]
    pages = [np.unique(s // PAGE) for s in seen]
    pool = sum(len(p) for p in pages) + spare
    order = rng.permutation(pool)
    table = np.full((B, blocks), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, p] = order[at:at + len(p)]
        at += len(p)
    live = np.zeros((pool, PAGE), bool)
    for b, s in enumerate(seen):
        live[table[b, s // PAGE], s % PAGE] = True
    d = dict(heads=heads, counts=list(counts), lens=list(lens), window=window, sinks=sinks,
             scale=float(scale), table=table, tokens=tokens, pool=pool,
             starts=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    rows = rng.standard_normal((pool, PAGE, D)).astype(np.float32)
    if fp8:
        from oracle import quantize_rows_fp8
        codes, exps = quantize_rows_fp8(rows.reshape(-1, D).astype(np.float64))
        codes, exps = codes.reshape(pool, PAGE, D).copy(), exps.reshape(pool, PAGE).copy()
        d["cache"] = fp8_values(codes, exps)
        codes[~live] = 0x7F  # NaN
        d["codes"], d["exps"] = codes, exps
    else:
        bits = bf16_bits(rows)
        d["cache"] = synth.bf16_bits_to_f64(bits)
        bits[~live] = 0x7FC0
        d["bits"] = bits
    q = bf16_bits(size * rng.standard_normal((tokens + pad, heads, D)).astype(np.float32))
    d["q"] = q
    return d


def fp8_values(codes, exps):
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9.0)
    return np.where(c & 128, -v, v) * 2.0 ** exps.astype(np.float64)[..., None]


def attention(d, only=None):
    """out, lse and the bounds of their errors, in 64 bits (of the tokens `only`, if given).

    A weight is rounded to bf16 (half a step), the sum over the weights is not; the scores'
    fp32 sums of 576 products are each off by at most 576 * 2^-23 of the sum of magnitudes,
    which moves a weight by twice that at most; exp2 and the scaling add under 1e-5; out is
    rounded to bf16 once."""
    q = synth.bf16_bits_to_f64(d["q"])
    T, H = q.shape[0], d["heads"]
    out, lse = np.zeros((T, H, D_C)), np.full((T, H), -np.inf)
    tol, ltol = np.zeros((T, H, D_C)), np.zeros((T, H))
    for b, (c, n) in enumerate(zip(d["counts"], d["lens"])):
        for i in range(c):
            t = int(d["starts"][b]) + i
            j = visible(n, c, i, d["window"], d["sinks"])
            if len(j) == 0 or (only is not None and t not in only):
                continue
            kv = d["cache"][d["table"][b, j // PAGE], j % PAGE]
            s = d["scale"] * q[t] @ kv.T
            off = 576 * 2.0 ** -23 * d["scale"] * (np.abs(q[t]) @ np.abs(kv).T).max(1)
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            z = w.sum(1, keepdims=True)
            w /= z
            out[t] = w @ kv[:, :D_C]
            lse[t] = (m + np.log(z))[:, 0]
            size = w @ np.abs(kv[:, :D_C])
            tol[t] = (HALF_STEP_BF16 + 2 * off[:, None] + 1e-5) * size + HALF_STEP_BF16 * (
                np.abs(out[t]) + HALF_STEP_BF16 * size) + 1e-30
            ltol[t] = off + 1e-5 * np.maximum(1, np.abs(lse[t]))
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what):
    assert got.shape == ref.shape, (got.shape, ref.shape)
    inf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: -inf pattern differs"
    err = np.abs(got[~inf] - ref[~inf])
    assert np.all(np.isfinite(err)), f"{what}: not finite"
    over = err - tol[~inf]
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over its bound"
