"""The 4-bit cache's format in 64 bits, from its definition, one row at a time."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every e4m3 number from 0 to 448, by its code
E4M3 = np.array([f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10) for e in range(16)
                 for f in range(8)][:127])


def nearest(x, numbers):
    """Index of the nearest of ascending numbers, the even index where two are equally near."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(numbers, x), 1, len(numbers) - 1)
    lo = hi - 1
    below, above = x - numbers[lo], numbers[hi] - x
    take = np.where(below == above, np.where(lo % 2 == 0, lo, hi), np.where(below < above, lo, hi))
    return np.where(x >= numbers[-1], len(numbers) - 1, take)


def quantize(rows):
    """Finite rows [n, 512] of bf16 values: codes [n, 512] (0..15), scales (codes) [n, 32], exps [n]."""
    rows = np.asarray(rows, np.float64)
    n = len(rows)
    most = np.abs(rows).max(1)
    exps = np.zeros(n, np.int64)
    for i, m in enumerate(most):
        if m > 0:
            e = -120
            while m > 2688.0 * 2.0 ** e:
                e += 1
            exps[i] = e
    x = rows / 2.0 ** exps[:, None].astype(np.float64)
    g = x.reshape(n, 32, 16)
    want = np.abs(g).max(2) / 6.0
    want = np.where(exps[:, None] == 117, np.minimum(want, 320.0), want)
    scales = nearest(want, E4M3)
    s = E4M3[scales][..., None]
    q = np.divide(np.abs(g), s, out=np.zeros_like(g), where=s > 0)
    codes = nearest(q, LEVELS)
    codes = codes + 8 * ((codes > 0) & (g < 0))  # zero has no sign
    return codes.reshape(n, 512), scales, exps


def values(codes, scales, exps):
    v = np.where(codes >= 8, -1.0, 1.0) * LEVELS[codes & 7]
    s = np.append(E4M3, np.nan)[scales & 127]
    with np.errstate(invalid="ignore"):
        v = v.reshape(len(codes), 32, 16) * s[..., None] * (2.0 ** exps.astype(np.float64))[:, None, None]
    return v.reshape(len(codes), 512)


def pack(codes):
    return (codes[..., ::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed):
    c = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), np.int64)
    c[..., ::2], c[..., 1::2] = packed & 15, packed >> 4
    return c
