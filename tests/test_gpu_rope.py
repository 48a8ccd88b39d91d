"""nvfp4_qk_norm_rope against the fp64 formula.

Tolerance, u = 2^-24: the mean of squares is off by (d / 16 + 8) u at most (16
terms in a lane, then up to 4 sums, quotient), its root by half that; with root,
quotient and two products the normed value is off by (d / 32 + 9) u of itself.  The
rotation adds two products and a sum: 3 u (|a| + |b|) of the pair.  Rounding to
bf16 adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from oracle import attn_ref as A
from tests.attn_util import i32
from tests.gpu_util import host_f32, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def run(T, hq, hk, d, rot, dtype, *, axes=1, adjacent=False, seed=0, gap=0, in_place=False, pos=None, pair_axis=None, spread=1.0):
    dev = need_gpu()
    print(f"[rope] T {T} heads {hq}/{hk}x{d} rot {rot} axes {axes} adjacent {adjacent} {dtype}", flush=True)
    rng = np.random.default_rng(seed)
    n_pos = 300
    q_col, k_col = gap, 2 * gap + hq * d
    x = torch.from_numpy((spread * rng.standard_normal((T, k_col + hk * d + gap))).astype(np.float32)).to(dev).to(dtype)
    if T > 2:
        x[1, q_col:q_col + d] = 0  # a head of zeros
    xh = host_f32(x).astype(np.float64)
    qw, kw = ((1 + 0.3 * rng.standard_normal(d)).astype(np.float32) for _ in range(2))
    angle = rng.uniform(-np.pi, np.pi, (n_pos, rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    if pos is None:
        pos = rng.integers(0, n_pos, (axes, T))
    pos = np.asarray(pos).reshape(axes, T)
    if axes > 1 and pair_axis is None:
        pair_axis = bytes(rng.integers(0, axes, rot // 2).astype(np.uint8))
    axis = np.zeros(rot // 2, int) if axes == 1 else np.frombuffer(pair_axis, np.uint8).astype(int)
    pt = torch.from_numpy(pos.astype(np.int32)).to(dev)
    q = x[:, q_col:q_col + hq * d] if in_place else torch.full((T, hq * d + gap), 7.5, dtype=BF, device=dev)
    k = x[:, k_col:k_col + hk * d] if in_place else torch.full((T, hk * d + gap), 7.5, dtype=BF, device=dev)
    got = nv.qk_norm_rope(x, torch.from_numpy(qw).to(dev), torch.from_numpy(kw).to(dev), torch.from_numpy(table).to(dev),
                          pt[0] if axes == 1 else pt, q_col=q_col, k_col=k_col, n_q_heads=hq, n_kv_heads=hk, eps=EPS,
                          pair_axis=pair_axis, adjacent=adjacent, q=q, k=k)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k
    known = np.all((pos >= 0) & (pos < n_pos), 0)
    at = np.where(known, pos, 0)[axis]                       # [pairs, T]
    cos, sin = (table[at, np.arange(rot // 2)[:, None] + o].T for o in (0, rot // 2))
    for name, y, w, col, heads in (("q", q, qw, q_col, hq), ("k", k, kw, k_col, hk)):
        xs = xh[:, col:col + heads * d].reshape(T, heads, d)
        want = A.norm_rope_ref(xs, w, EPS, cos, sin, adjacent) * known[:, None, None]
        size = A.norm_rope_ref(xs, w, EPS, np.ones_like(cos), np.zeros_like(sin), adjacent)
        turn = np.abs(size)
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, rot // 2 + i)
        both = turn[..., a] + turn[..., b]
        turn = np.abs(size).copy()
        turn[..., a] = turn[..., b] = both
        tol = (d / 32 + 12) * U * turn + 2.0 ** -8 * np.abs(want) + 2.0 ** -126
        g = host_f32(y).astype(np.float64)
        err = np.abs(g[:, :heads * d].reshape(want.shape) - want)
        assert np.all(err <= tol), f"{name}: {np.count_nonzero(err > tol)} off, worst {np.max(err / tol)}"
        assert np.all(g[~known][:, :heads * d] == 0.0)
        if not in_place:
            assert np.all(g[:, heads * d:] == 7.5)
    if in_place:
        h = host_f32(x).astype(np.float64)
        for lo, hi in ((0, q_col), (q_col + hq * d, k_col), (k_col + hk * d, x.shape[1])):
            assert np.array_equal(h[:, lo:hi], xh[:, lo:hi])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 24, 4, 256, 64), (3, 1, 1, 64, 64), (70, 32, 8, 128, 128), (33, 5, 1, 128, 16),
                                           (9, 3, 2, 64, 48), (257, 6, 2, 256, 256), (5000, 2, 1, 64, 32)])
def test_heads_and_sizes(T, hq, hk, d, rot, adjacent, dtype):
    run(T, hq, hk, d, rot, dtype, adjacent=adjacent, seed=T + d, gap=8)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("adjacent", [False, True])
def test_several_axes(axes, adjacent):
    run(131, 6, 2, 128, 96, BF, axes=axes, adjacent=adjacent, seed=axes)
    run(7, 3, 1, 256, 256, F32, axes=axes, adjacent=adjacent, seed=axes)


def test_positions_outside_the_table_give_zeros():
    pos = np.array([0, -1, 299, 300, 2 ** 31 - 1, -2 ** 31, 5])
    run(7, 4, 2, 64, 32, BF, pos=pos)
    both = np.stack([np.arange(7), pos])
    run(7, 4, 2, 64, 32, BF, axes=2, pos=both, pair_axis=bytes(16))  # an axis that no pair uses counts too


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place(adjacent):
    run(67, 5, 2, 128, 64, BF, adjacent=adjacent, gap=16, in_place=True)


@pytest.mark.parametrize("spread", [1e-4, 1e15])
def test_sizes_of_values(spread):
    """Rows whose mean square lies near eps, or near the top of fp32."""
    run(20, 3, 1, 128, 64, F32, spread=spread)


def test_what_is_not_finite_stays_in_its_head():
    dev = need_gpu()
    print("[rope] non-finite", flush=True)
    x = torch.ones((3, 4 * 64), device=dev)
    x[1, 64 + 3] = float("nan")
    x[2, 2 * 64] = float("inf")
    w = torch.ones(64, device=dev)
    table = torch.cat([torch.ones((4, 16)), torch.zeros((4, 16))], 1).to(dev)
    q, k = nv.qk_norm_rope(x, w, w, table, i32([0, 1, 2], dev), q_col=0, k_col=128, n_q_heads=2, n_kv_heads=2)
    torch.cuda.synchronize()
    bad_q, bad_k = torch.isnan(q.reshape(3, 2, 64)).any(-1).cpu(), torch.isnan(k.reshape(3, 2, 64)).any(-1).cpu()
    assert bad_q.tolist() == [[False, False], [False, True], [False, False]]
    assert bad_k.tolist() == [[False, False], [False, False], [True, False]]


def test_stream_and_graph():
    dev = need_gpu()
    print("[rope] stream and graph", flush=True)
    x = torch.randn((12, 8 * 64), device=dev).to(BF)
    w = torch.rand(64, device=dev)
    table = torch.randn((50, 64), device=dev)
    pos = i32(range(12), dev)
    args = dict(q_col=0, k_col=6 * 64, n_q_heads=6, n_kv_heads=2)
    want = nv.qk_norm_rope(x, w, w, table, pos, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.qk_norm_rope(x, w, w, table, pos, stream=side, **args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    q, k = (torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.qk_norm_rope(x, w, w, table, pos, q=q, k=k, **args)
    for shift in (0, 7, 38):
        pos.copy_(i32(range(shift, shift + 12), dev))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, k), nv.qk_norm_rope(x, w, w, table, pos, **args)))
