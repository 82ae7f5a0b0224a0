"""The training operators' definitions in 64 bits (numpy), written from include/demo.h alone."""

import numpy as np

BLOCK = 128
_M = (1 << 64) - 1


def sm(z):
    z = (z + 0x9E3779B97F4A7C15) & _M
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & _M
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & _M
    return z ^ (z >> 31)


def threshold(p):
    return int(np.rint(65536.0 * p))


def keep_mask(rows, cols, p, seed, step, site):
    """Bool [rows, cols], one element at a time in Python integers."""
    T, G = threshold(p), (cols + 3) // 4
    key = sm(sm(sm(seed) ^ step) ^ site)
    out = np.zeros((rows, cols), dtype=bool)
    for r in range(rows):
        for g in range(G):
            h = sm(key ^ (r * G + g))
            for e in range(min(4, cols - 4 * g)):
                out[r, 4 * g + e] = ((h >> (16 * e)) & 0xFFFF) >= T
    return out


def drop_scale(p):
    T = threshold(p)
    return 65536.0 / (65536.0 - T) if T < 65536 else 0.0


def dropout(x, p, seed, step, site, residual=None):
    keep = keep_mask(*x.shape, p, seed, step, site)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(keep, x.astype(np.float64) * drop_scale(p), 0.0)
    return y if residual is None else y + residual.astype(np.float64), keep


LIMITS = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def block_scale(values, fmt):
    """The block's scale, searched from the definition."""
    v = np.abs(values[np.isfinite(values)])
    amax = v.max() if v.size else 0.0
    if amax == 0.0:
        return 1.0
    e = -126
    while amax > 2.0 ** e * LIMITS[fmt][2]:
        e += 1
    return 2.0 ** e


def round_code(v, fmt):
    """Nearest representable value of the format, ties to the even significand."""
    mant, least, top = LIMITS[fmt]
    if not np.isfinite(v):
        return np.nan
    if v == 0.0:
        return 0.0
    grain = 2.0 ** (max(int(np.floor(np.log2(abs(v)))), least) - mant)
    r = np.rint(v / grain) * grain
    assert abs(r) <= top
    return r


def quantize(x, fmt, tiles=False):
    """(codes [rows, kp], scales [kb, rows]) by rows, as float64 values."""
    rows, k = x.shape
    kb = (k + BLOCK - 1) // BLOCK
    codes, scales = np.zeros((rows, kb * BLOCK)), np.ones((kb, rows))
    for b in range(kb):
        cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        for r in range(rows):
            t = r // BLOCK * BLOCK
            scales[b, r] = block_scale(x[t:t + BLOCK, cols] if tiles else x[r, cols], fmt)
            codes[r, cols] = [round_code(v / scales[b, r], fmt) for v in x[r, cols]]
    return codes, scales


def values(codes, scales, k):
    rows = codes.shape[0]
    return (codes * np.repeat(scales[:, :rows].T, BLOCK, axis=1))[:, :k]


def product(av, bv):
    """(a b^T, sum |a||b|) in 64 bits."""
    return av @ bv.T, np.abs(av) @ np.abs(bv).T


def product_tolerance(total, k):
    """Elementwise bound of a product's float32 sums: over at most 512 of k, sixteen instructions
    that each align 32 products and the running sum to the largest term and may drop what is below
    2^-24 of it (33 terms each); over the longer sum, an addition for each 512, within 2^-24."""
    return (16 * 33 + (k + 511) // 512) * 2.0 ** -24 * total


def round_tolerance(want, dtype):
    """Half a unit in the last place of the output's type (float16's smallest steps included)."""
    bits, tiny = {"f32": (24, 0.0), "bf16": (8, 0.0), "f16": (11, 2.0 ** -25)}[dtype]
    return np.abs(want) * 2.0 ** -bits + tiny
