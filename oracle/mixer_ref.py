"""References of the operators around the GDN projections: plain numpy fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): imported by tests,
never by the product path.  The recurrence itself is ``gdn_ref``'s, run here
sequence by sequence; the short convolution and the norms are written out
from their formulas.
"""
from __future__ import annotations

import numpy as np

from .gdn_ref import gdn_recurrence_ref, l2_normalize


def silu(x):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def gdn_packed_ref(q, k, v, g, beta, cu, starts=None):
    """The recurrence over packed sequences cu[i] .. cu[i + 1] - 1.  starts:
    per sequence a state [n_v, d, d] or None.  Returns (o [rows, n_v, d_v] with
    zeros outside the sequences, final states [n_seqs, n_v, d, d], |S_t|_F
    [rows, n_v])."""
    n, n_v, d = len(cu) - 1, v.shape[1], v.shape[2]
    o, norms = np.zeros(v.shape), np.zeros(v.shape[:2])
    states = np.zeros((n, n_v, q.shape[2], d))
    for i in range(n):
        a, b = int(cu[i]), int(cu[i + 1])
        s0 = None if starts is None else starts[i]
        if b <= a:
            states[i] = 0.0 if s0 is None else s0
            continue
        o[a:b], states[i], _, nr = gdn_recurrence_ref(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], s0=s0)
        norms[a:b] = np.sqrt(nr)
    return o, states, norms


def conv_silu_ref(x, w, cu, old):
    """y_t = silu(sum_i w[:, i] x_{t - W + 1 + i}) per sequence, whose rows are
    preceded by old[i] [W - 1, channels].  Returns (y, the magnitude sum
    sum_i |w x| before the SiLU, the new states)."""
    x, w, old = (np.asarray(t, dtype=np.float64) for t in (x, w, old))
    width = w.shape[1]
    y, mag, new = np.zeros_like(x), np.zeros_like(x), old.copy()
    for s in range(len(cu) - 1):
        a, b = int(cu[s]), int(cu[s + 1])
        rows = np.concatenate([old[s], x[a:b]])
        for t in range(b - a):
            y[a + t] = np.sum(rows[t:t + width] * w.T, axis=0)
            mag[a + t] = np.sum(np.abs(rows[t:t + width] * w.T), axis=0)
        new[s] = rows[len(rows) - (width - 1):]
    return silu(y), mag, new


def add_rmsnorm_ref(x, residual, scale, w, eps):
    """(t, y, mean square) of t = residual + scale x and y = t / sqrt(mean t^2 + eps) w."""
    x = np.asarray(x, dtype=np.float64)
    t = scale * x + (0.0 if residual is None else np.asarray(residual, dtype=np.float64))
    ms = np.mean(t * t, axis=-1, keepdims=True)
    return t, t / np.sqrt(ms + eps) * np.asarray(w, dtype=np.float64), ms


def rmsnorm_gated_ref(o, z, w, eps):
    """y of rmsnorm_gated: groups of len(w) columns of o, times w, times silu(z)."""
    o, z = np.asarray(o, dtype=np.float64), np.asarray(z, dtype=np.float64)
    w = np.asarray(w, dtype=np.float64)
    g = o.reshape(o.shape[0], -1, len(w))
    y = g / np.sqrt(np.mean(g * g, axis=-1, keepdims=True) + eps) * w
    return y.reshape(o.shape) * silu(z)


__all__ = ["silu", "gdn_packed_ref", "conv_silu_ref", "add_rmsnorm_ref", "rmsnorm_gated_ref", "l2_normalize"]
