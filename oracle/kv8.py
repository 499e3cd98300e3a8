"""The 8-bit K/V cache (TEST INFRASTRUCTURE, see the package docstring): E4M3
codes with one power-of-two scale per block of 32 tokens, float64.

One sequence and KV head at a time, positions in order (no pages).  A block's
scale is the least 2^e, e >= -126, with |x| <= 448 * 2^e over its new finite
rows, or the old scale if that is larger and older rows are in the block; new
rows are stored as the nearest code of x / scale (ties to even, saturating),
older rows are brought to the scale in the same way.
"""
import numpy as np

from .quant import e4m3_decode, round_e4m3

BLOCK = 32


def scale_for(x):
    x = np.abs(np.asarray(x, dtype=np.float64))
    a = float(np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0))
    if a == 0.0:
        return 2.0 ** -126
    f, e = np.frexp(a)                       # a = f * 2^e, f in [0.5, 1)
    return 2.0 ** max(-126, int(e) - 9 + (f > 0.875))


def encode(x):
    """Nearest E4M3 codes; NaN is code 0x7f with the sign of x."""
    x = np.asarray(x, dtype=np.float64)
    c = round_e4m3(np.clip(np.nan_to_num(x, nan=0.0, posinf=448, neginf=-448),
                           -448, 448))
    return np.where(np.isnan(x), 0x7F, c).astype(np.uint8)


def append(codes, scales, pos, rows):
    """Append rows [n, hd] at position pos: codes uint8 [cap, hd] and scales
    [cap / 32] are changed in place."""
    end = pos + len(rows)
    for j in range(pos // BLOCK, -(-end // BLOCK) if len(rows) else 0):
        p0 = j * BLOCK
        lo, hi = max(pos, p0), min(end, p0 + BLOCK)
        x = np.asarray(rows[lo - pos:hi - pos], dtype=np.float64)
        s = scale_for(x)
        if lo > p0:
            s = max(s, scales[j])
            if s != scales[j]:
                codes[p0:lo] = encode(e4m3_decode(codes[p0:lo]) * (scales[j] / s))
        codes[lo:hi] = encode(x / s)
        scales[j] = s


def decode(codes, scales, n):
    """The first n rows' values."""
    return e4m3_decode(codes[:n]) * np.repeat(scales, BLOCK)[:n, None]


def attend(q, k, v, window, scale):
    """One query's heads q [G, hd] over the rows k, v [n, hd]; also the
    attention average of |v| (what relative errors of the weights act on).
    No rows: zeros."""
    n = len(k)
    lo = max(0, n - window) if window else 0
    if n == 0:
        return np.zeros(q.shape), np.zeros(q.shape)
    z = scale * (np.asarray(q, np.float64) @ k[lo:].T)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ v[lo:], p @ np.abs(v[lo:])
