"""References of the attention layer's operators: plain numpy fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): imported by tests,
never by the product path.  Written from the formulas: the norm and rotation
per head, the two cache formats byte by byte, and the attention row by row.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4_ref as ref


def norm_rope_ref(x, w, eps, cos, sin, adjacent):
    """x [T, heads, d], w [d]; cos and sin [T, pairs], the angle of each pair.
    Returns the normed and turned heads."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    half = cos.shape[1]
    c, s = (np.asarray(t, dtype=np.float64)[:, None] for t in (cos, sin))
    out = y.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, half + i)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def e4m3_codes(x, g):
    """E4M3 bytes of x / g: round to nearest even of the exact quotient,
    saturated at 448, 0x7F for what is not finite.  The quotient is compared with
    the midpoints as x against midpoint * g, exact in fp64."""
    x = np.asarray(x, dtype=np.float64)
    g = float(g)
    mid = ref.E4M3_MIDPOINTS * g
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(lo == hi, lo, lo + lo % 2)   # on midpoint lo, between codes lo and lo + 1: the even one
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def e4m3_values(codes):
    codes = np.asarray(codes)
    table = np.concatenate([ref.E4M3_VALUES, [np.nan]])
    return np.where(codes & 0x80, -1.0, 1.0) * table[codes & 0x7F]


def kv_values(fmt, codes, scales, g):
    """Values of rows of codes [..., d] (fp8) or [..., d / 2] with scales [..., d / 16]."""
    if fmt == "fp8":
        return e4m3_values(codes) * float(g)
    codes = np.asarray(codes)
    pair = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(pair & 8, -1.0, 1.0) * ref.E2M1_VALUES[pair & 7]
    return v * np.repeat(e4m3_values(scales), 16, -1) * float(g)


def seen_ref(n, kv, n_keys, tree=None):
    """[n, n_keys]: which positions the rows of a sequence of length kv see."""
    p, j = np.arange(n_keys)[None], np.arange(n)[:, None]
    if tree is None:
        s = p <= kv - n + j
    else:
        bit = p - (kv - n)
        word = np.asarray(tree, dtype=np.int64).astype(np.uint64)[:, None]
        s = (bit < 0) | ((bit < 64) & ((word >> np.clip(bit, 0, 63).astype(np.uint64)) & np.uint64(1) == 1))
    return s & (p < kv)


def attn_ref(q, k, v, seen, scale):
    """q [n, hq, d], k and v [keys, hk, d], seen [n, keys].  Returns (o [n, hq,
    d], sum w |v| / sum w, largest sum |q k| scale of a row, sum |v|).  What is not
    seen counts for nothing, whatever it is; a row that sees nothing is zeros."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq, d = q.shape
    group = hq // k.shape[1]
    o, mag, flat, big = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), np.zeros((n, hq))
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        for i in range(n):
            at = seen[i]
            if not at.any():
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                s = kh[at] @ q[i, h] * scale
                w = np.exp(s - np.max(s))
                w /= w.sum()
                o[i, h], mag[i, h], flat[i, h] = w @ vh[at], w @ np.abs(vh[at]), np.abs(vh[at]).sum(0)
                big[i, h] = np.max(np.abs(kh[at]) @ np.abs(q[i, h])) * scale
    return o, mag, big, flat
