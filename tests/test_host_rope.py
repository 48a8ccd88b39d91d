"""nvfp4_qk_norm_rope's kernel in a build for the host (tests/host_wave): accesses, and results against the fp64 formula
within tests/test_gpu_rope.py's bound."""
import numpy as np
import pytest

from oracle import attn_ref as A
from tests import host_wave as H

U = 2.0 ** -24
EPS = 1e-6


def check(lib, T, hq, hk, d, rot, *, bf16, spread, axes=1, adjacent=False, at_end=True, seed=0):
    rng = np.random.default_rng(seed)
    n_pos, gap = 40, 8
    q_col, k_col = gap, 2 * gap + hq * d
    x = (np.asarray(spread).reshape(-1, 1) * rng.standard_normal((T, k_col + hk * d))).astype(np.float32)
    given = H.bf16(x) if bf16 else x
    xh = (H.f32(given) if bf16 else x).astype(np.float64)
    qw, kw = ((1 + 0.3 * rng.standard_normal(d)).astype(np.float32) for _ in range(2))
    angle = rng.uniform(-np.pi, np.pi, (n_pos, rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = rng.integers(0, n_pos, (axes, T))
    axis = rng.integers(0, axes, rot // 2)
    got = H.rope(lib, given, qw, kw, table, pos, q_col=q_col, k_col=k_col, hq=hq, hk=hk, eps=EPS,
                 pair_axis=axis.tolist() if axes > 1 else None, adjacent=adjacent, at_end=at_end)
    at = pos[axis]
    cos, sin = (table[at, np.arange(rot // 2)[:, None] + o].T for o in (0, rot // 2))
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, rot // 2 + i)
    for y, w, col, heads in ((got[0], qw, q_col, hq), (got[1], kw, k_col, hk)):
        xs = xh[:, col:col + heads * d].reshape(T, heads, d)
        want = A.norm_rope_ref(xs, w, EPS, cos, sin, adjacent)
        turn = np.abs(A.norm_rope_ref(xs, w, EPS, np.ones_like(cos), np.zeros_like(sin), adjacent))
        both = turn[..., a] + turn[..., b]
        turn[..., a] = turn[..., b] = both
        tol = (d / 32 + 12) * U * turn + 2.0 ** -8 * np.abs(want) + 2.0 ** -126
        err = np.abs(y.reshape(want.shape) - want)
        assert np.all(err <= tol), f"{np.count_nonzero(~(err <= tol))} of {err.size} off"


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,axes,adjacent", [(3, 5, 2, 64, 48, 1, False), (1, 24, 4, 256, 64, 1, False),
                                                         (9, 3, 1, 128, 128, 3, True), (5, 1, 1, 256, 16, 2, True)])
@pytest.mark.parametrize("at_end", [True, False])
def test_bounds_and_values(host_lib, T, hq, hk, d, rot, axes, adjacent, bf16, at_end):
    check(host_lib, T, hq, hk, d, rot, bf16=bf16, spread=1.0, axes=axes, adjacent=adjacent, at_end=at_end)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_squares_past_fp32(host_lib, d, bf16):
    """Finite heads whose sum of squares is not, beside ordinary ones, up to the top of fp32."""
    spread = [1.0, 1e14, 3e15, 1e16, 1e18, 3e18, 1e19, 1e25, 7e37, 1e-3]
    check(host_lib, len(spread), 3, 2, d, 32, bf16=bf16, spread=spread)
