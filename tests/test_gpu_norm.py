"""nvfp4_add_rmsnorm and nvfp4_rmsnorm_gated against the fp64 formulas.

Tolerances, in units of u = 2^-24 (one fp32 rounding).  add_rmsnorm: t is one
fused rounding of residual + scale x, off by at most u (|residual| + |scale x|)
=: u m.  The sum of squares adds at most 16 terms in a lane, then 6 + 16
partial sums, each term off by 2 u m |t|, so mean t^2 is off by at most
(40 + 2 kappa) u of itself with kappa = |m| / |t| (norms of the row); its root
by half that, and three further roundings (root, quotient, two products) end at
|y - Y| <= u ((26 + kappa) |Y| + m w / rms).  rmsnorm_gated: o enters exactly
(kappa = 1, no m term), and silu's exp2 argument is off by u |z| log2(e), its
exp2, sum and reciprocal by 4 u together: |y - Y| <= u (34 + 2 |z|) |Y|.  bf16
output adds half a bf16 ulp, 2^-8 of the value; a bf16 t likewise.  Values
below the fp32 normal range may flush: 2^-120 absolute."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from oracle import mixer_ref as M
from tests.gpu_util import host_f32, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def _padded(a, dtype, pad, dev):
    """a as a view of rows that are `pad` columns longer (NaN between the rows)."""
    buf = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=dtype, device=dev)
    buf[:, :a.shape[1]] = torch.from_numpy(a).to(dev).to(dtype)
    return buf[:, :a.shape[1]]


def _close(got, want, tol, what):
    g = host_f32(got).astype(np.float64)
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    bad = np.argwhere(~(np.abs(g - want) <= tol + 2.0 ** -120))
    assert bad.size == 0, f"{what}: {len(bad)} out of tolerance, first {bad[0].tolist()}: " \
                          f"{g[tuple(bad[0])]!r} vs {want[tuple(bad[0])]!r} (tol {tol[tuple(bad[0])]!r})"


def _check_add(rows, cols, xd, rd, od, scale, seed, *, residual=True, pad=0, in_place=False, outlier=0.0):
    dev = need_gpu()
    print(f"[add_norm] {rows}x{cols} x {xd} r {rd} y {od} pad {pad}", flush=True)
    rng = np.random.default_rng(seed)
    x = _padded(rng.standard_normal((rows, cols)).astype(np.float32), xd, pad, dev)
    r = rng.standard_normal((rows, cols)).astype(np.float32)
    if outlier:
        r[:, cols // 2] = outlier
    r = _padded(r, rd, pad, dev) if residual else None
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(cols)).astype(np.float32)).to(dev)
    xh, rh = host_f32(x), host_f32(r) if residual else np.zeros((rows, cols), np.float32)
    s = r if in_place else torch.full((rows, cols + pad), float("nan"), dtype=rd, device=dev)[:, :cols]
    y = torch.full((rows, cols + pad), float("nan"), dtype=od, device=dev)
    got = nv.add_rmsnorm(x, w, residual=r, scale=scale, eps=EPS, residual_out=s, out=y)
    assert got is y
    torch.cuda.synchronize()
    sc = float(np.float32(scale))
    t, Y, ms = M.add_rmsnorm_ref(xh, rh, sc, w.cpu().numpy(), float(np.float32(EPS)))
    m = np.abs(rh.astype(np.float64)) + np.abs(sc * xh.astype(np.float64))
    kappa = np.linalg.norm(m, axis=1, keepdims=True) / np.maximum(np.linalg.norm(t, axis=1, keepdims=True), 1e-300)
    inv = np.abs(w.cpu().numpy()) / np.sqrt(ms + EPS)
    _close(y[:, :cols], Y, U * ((26 + kappa) * np.abs(Y) + m * inv), "y")
    _close(s, t, U * m, "t")
    if pad:
        assert torch.isnan(y[:, cols:].float()).all(), "y written past its columns"


@pytest.mark.parametrize("rows,cols,xd,rd,od", [
    (1, 5120, F32, F32, BF), (3, 5120, BF, BF, BF), (7, 4096, BF, F32, F32), (2, 16384, BF, BF, BF),
    (5, 16, F32, BF, F32), (33, 1040, BF, BF, F32), (300, 512, BF, BF, BF)])
def test_add_rmsnorm_aligned(rows, cols, xd, rd, od):
    _check_add(rows, cols, xd, rd, od, 0.7, rows + cols)


@pytest.mark.parametrize("rows,cols,xd,rd,od,pad", [
    (4, 1, BF, BF, F32, 0), (3, 17, F32, F32, BF, 2), (9, 1023, BF, F32, BF, 0), (2, 16383, BF, BF, BF, 0),
    (6, 1024, BF, BF, F32, 3), (6, 1024, BF, BF, BF, 16), (5, 321, F32, BF, F32, 1)])
def test_add_rmsnorm_odd_columns_and_strides(rows, cols, xd, rd, od, pad):
    _check_add(rows, cols, xd, rd, od, -1.25, rows * 7 + cols, pad=pad)


def test_add_rmsnorm_in_place_no_residual_and_outliers():
    _check_add(8, 5120, BF, BF, BF, 1.0, 1, in_place=True)
    _check_add(8, 999, BF, BF, F32, 1.0, 2, in_place=True)
    _check_add(8, 2048, BF, F32, F32, 0.5, 3, residual=False)
    _check_add(8, 2048, BF, F32, F32, 1.0, 4, outlier=3.0e4)


def test_add_rmsnorm_zero_rows_and_empty():
    dev = need_gpu()
    x = torch.zeros((3, 256), dtype=BF, device=dev)
    w = torch.ones(256, device=dev)
    y = nv.add_rmsnorm(x, w, residual=x, residual_out=torch.empty_like(x))
    assert torch.equal(y, torch.zeros_like(y))                    # eps keeps a zero row finite
    assert nv.add_rmsnorm(x[:0], w).shape == (0, 256)
    # a row with an infinity or a NaN leaves the others as they are
    x = torch.randn((4, 256), device=dev).to(BF)
    want = nv.add_rmsnorm(x, w).clone()
    x[1, 3], x[2, 200] = float("inf"), float("nan")
    got = nv.add_rmsnorm(x, w)
    assert torch.equal(got[[0, 3]], want[[0, 3]])
    assert torch.isnan(got[1, 3]) and torch.isnan(got[2]).all()


def _check_gated(rows, heads, group, od_in, zd, od, seed, pad=0, big=1.0):
    dev = need_gpu()
    print(f"[gated] {rows}x{heads}x{group} o {od_in} z {zd} y {od} pad {pad}", flush=True)
    rng = np.random.default_rng(seed)
    cols = heads * group
    o = _padded((rng.standard_normal((rows, cols)) * 0.1).astype(np.float32), od_in, pad, dev)
    z = _padded((rng.standard_normal((rows, cols)) * big).astype(np.float32), zd, pad, dev)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(group)).astype(np.float32)).to(dev)
    y = torch.full((rows, cols + pad), float("nan"), dtype=od, device=dev)
    nv.rmsnorm_gated(o, z, w, eps=EPS, out=y)
    torch.cuda.synchronize()
    Y = M.rmsnorm_gated_ref(host_f32(o), host_f32(z), w.cpu().numpy(), float(np.float32(EPS)))
    _close(y[:, :cols], Y, U * (34 + 2 * np.abs(host_f32(z).astype(np.float64))) * np.abs(Y), "y")
    if pad:
        assert torch.isnan(y[:, cols:].float()).all(), "y written past its columns"


@pytest.mark.parametrize("rows,heads,group,od_in,zd,od,pad", [
    (1, 32, 128, BF, BF, BF, 0), (5, 32, 128, BF, BF, F32, 64), (3, 1, 16, F32, F32, F32, 0),
    (7, 3, 32, BF, F32, BF, 8), (2, 5, 64, F32, BF, F32, 0), (9, 7, 256, BF, BF, BF, 24), (3, 2, 512, BF, BF, F32, 0),
    (5, 3, 1024, F32, F32, BF, 0), (257, 11, 128, BF, BF, BF, 0)])
def test_rmsnorm_gated(rows, heads, group, od_in, zd, od, pad):
    _check_gated(rows, heads, group, od_in, zd, od, rows + heads * group, pad=pad)


def test_rmsnorm_gated_wide_gates_and_empty():
    _check_gated(6, 4, 128, BF, F32, F32, 9, big=60.0)            # silu far into both of its tails
    dev = need_gpu()
    z = torch.zeros((0, 256), dtype=BF, device=dev)
    assert nv.rmsnorm_gated(z, z, torch.ones(128, device=dev)).shape == (0, 256)


@pytest.mark.parametrize("rows,cols", [(1, 5120), (37, 4096), (5, 16)])
def test_quantized_output_is_the_quantizer_of_the_fp32_output(rows, cols):
    """Codes and block scales equal nvfp4_quantize's of the fp32 y of the same
    call, with and without the values beside them, for both norms."""
    dev = need_gpu()
    print(f"[norm codes] {rows}x{cols}", flush=True)
    g = torch.Generator(device=dev).manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g, device=dev).to(BF)
    z = torch.randn((rows, cols), generator=g, device=dev).to(BF)
    gs = torch.tensor([0.0021], device=dev)
    w = torch.rand(cols, generator=g, device=dev) + 0.5
    wg = torch.rand(16, generator=g, device=dev) + 0.5
    for f in (lambda **k: nv.add_rmsnorm(x, w, residual=z, y_gs=gs, **k),
              lambda **k: nv.rmsnorm_gated(x, z, wg, y_gs=gs, **k)):
        y, codes, scales = f(out_dtype=F32)
        qc, qs, _ = nv.quantize(y, gs, from_amax=False)
        assert torch.equal(codes, qc) and torch.equal(scales, qs)
        none, c2, s2 = f()
        assert none is None and torch.equal(c2, qc) and torch.equal(s2, qs)


def test_rows_past_32_bit_offsets():
    """More than 2^31 values in front of the last rows."""
    dev = need_gpu()
    rows, cols = (1 << 17) + 3, 16384
    print(f"[norm] {rows}x{cols} bf16", flush=True)
    x = torch.empty((rows, cols), dtype=BF, device=dev)
    x[-3:] = torch.randn((3, cols), device=dev).to(BF)
    w = torch.ones(cols, device=dev)
    y = torch.empty_like(x)
    nv.add_rmsnorm(x, w, out=y)
    assert torch.equal(y[-3:], nv.add_rmsnorm(x[-3:].contiguous(), w))
    wg = torch.ones(1024, device=dev)
    nv.rmsnorm_gated(x, x, wg, out=y)
    tail = x[-3:].contiguous()
    assert torch.equal(y[-3:], nv.rmsnorm_gated(tail, tail, wg))


def test_refusals():
    dev = need_gpu()
    x, w = torch.zeros((2, 256), dtype=BF, device=dev), torch.ones(256, device=dev)
    gs = torch.ones(1, device=dev)
    for bad in (lambda: nv.add_rmsnorm(x.half(), w), lambda: nv.add_rmsnorm(x.t(), w),
                lambda: nv.add_rmsnorm(x, w[:-1]), lambda: nv.add_rmsnorm(x, w.to(BF)),
                lambda: nv.add_rmsnorm(x, w, residual=x[:1]), lambda: nv.add_rmsnorm(x.cpu(), w),
                lambda: nv.add_rmsnorm(x, w, residual=x, residual_out=x.float()),
                lambda: nv.add_rmsnorm(x, w, out=x[:1]), lambda: nv.add_rmsnorm(x, w, codes=x.byte()),
                lambda: nv.add_rmsnorm(x[:, :24], w[:24].contiguous(), y_gs=gs),
                lambda: nv.rmsnorm_gated(x, x[:, :128], w[:128]), lambda: nv.rmsnorm_gated(x, x, w.to(BF))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.rmsnorm_gated(x, x, w[:48].contiguous()), lambda: nv.add_rmsnorm(x, w, eps=0.0),
                lambda: nv.add_rmsnorm(x, w, scale=float("nan")),
                lambda: nv.rmsnorm_gated(x[:, 8:136], x[:, 1:129], w[:128].contiguous())):
        with pytest.raises(nv.Nvfp4Error):
            bad()


@pytest.mark.parametrize("cols", [15, 18, 31, 33, 100, 511, 1009, 1025, 1039, 5119])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_rmsnorm_rows_that_end_inside_a_lane(cols, dtype):
    """The last lane takes values that the lane before it has too, of which it may already have written the sum."""
    _check_add(5, cols, dtype, dtype, dtype, 0.5, cols, pad=1)
    _check_add(70, cols, dtype, dtype, BF, 1.0, cols + 1, in_place=True)
