"""The 8-bit K/V cache (TEST INFRASTRUCTURE, see the package docstring): E4M3
codes with one power-of-two scale per block of 32 tokens, float64.

One sequence and KV head at a time, positions in order (no pages).  A block's
scale is the least 2^e, e >= -126, with |x| <= 448 * 2^e over its new finite
rows, or the old scale if that is larger and older rows are in the block; new
rows are stored as the nearest code of x / scale (ties to even, saturating),
older rows are brought to the scale in the same way.
"""
import numpy as np

from .model import DT, Model
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


def round_bf16(x):
    """Nearest bf16 values, ties to even (finite x)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(DT)


class Kv8Model(Model):
    """The looped model whose full-attention layers hold their K/V in 8 bits:
    a call's rows (rounded to bf16, what a bf16 cache holds) are appended to
    the layer's codes, then every query reads the decoded values.  jitter:
    relative size of a random change of every k and v before they are stored,
    to measure how much the stored codes depend on it."""

    def __init__(self, *args, jitter=0.0, **kw):
        super().__init__(*args, **kw)
        self.codes, self.jitter = {}, jitter
        self.rng = np.random.default_rng(99)

    def store_kv(self, i, slot, pos, k, v):
        K, V = super().store_kv(i, slot, pos, k, v)
        if self.shape.layer_types[i] != 1:
            return K, V
        end = int(pos[-1]) + 1
        cap = -(-end // BLOCK) * BLOCK
        for kind, (x, out) in enumerate(((k, K), (v, V))):
            x = x * (1 + self.jitter * self.rng.uniform(-1, 1, x.shape))
            for b in range(x.shape[0]):
                for h in range(x.shape[1]):
                    c, s = self.codes.get((i, slot, kind, b, h),
                                          (np.zeros((0, x.shape[-1]), np.uint8),
                                           np.zeros(0)))
                    if len(c) < cap:
                        c = np.concatenate([c, np.zeros((cap - len(c), c.shape[1]), np.uint8)])
                        s = np.concatenate([s, np.zeros(cap // BLOCK - len(s))])
                    self.codes[i, slot, kind, b, h] = c, s
                    append(c, s, int(pos[0]), round_bf16(x[b, h]))
                    out[b, h, :end] = decode(c, s, end)
        return K, V
