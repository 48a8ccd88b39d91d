"""Outputs in the place of inputs, and in other columns of the rows that hold
them, where the GDN mixer's calls allow it: the bits of the same call with
memory of its own.  And refusals of real tensors that lie on each other."""
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import need_gpu
from tests.test_gpu_gdn_serve import BF, D, F32, _cu, _tensors

pytestmark = pytest.mark.gpu


def _rows(rows, cols, dtype, seed):
    dev = need_gpu()
    return torch.randn((rows, cols), generator=torch.Generator(device=dev).manual_seed(seed), device=dev).to(dtype)


@pytest.mark.parametrize("n_qk,n_v,many", [(1, 2, 1), (2, 4, 60), (1, 8, 70)])
def test_outputs_in_other_columns_of_the_input_rows(n_qk, n_v, many):
    print(f"[overlap] heads {n_qk}/{n_v}, {many} sequences", flush=True)
    T = 3 * many + 130
    x, gates, lay = _tensors(T, n_qk, n_v, many)
    cu = torch.tensor([3 * i for i in range(many)] + [T], dtype=torch.int32, device=x.device)
    w, width = x.shape[1], n_v * D
    s = torch.zeros((T, n_v, D, D), device=x.device)
    for f in (lambda x, **k: nv.gdn_prefill(x, gates, cu, **lay, **k), lambda x, **k: nv.gdn_decode(x, gates, s.zero_(), **lay, **k)):
        rows = torch.full((T, w + width + 8), float("nan"), dtype=BF, device=x.device)
        rows[:, :w] = x
        want = f(x)
        f(rows, o=rows[:, w + 8:])
        assert torch.equal(rows[:, w + 8:], want) and torch.equal(rows[:, :w], x) and rows[:, w:w + 8].isnan().all()


@pytest.mark.parametrize("channels,dtype,step", [(64, BF, False), (13, F32, False), (1025, F32, True), (2056, BF, True)])
def test_convolution_into_other_columns(channels, dtype, step):
    print(f"[overlap] convolution {channels} {dtype} step {step}", flush=True)
    rows = _rows(70, 2 * channels + 3, dtype, channels)
    w = _rows(channels, 4, F32, 1)
    x, y = rows[:, :channels], rows[:, channels + 3:]
    cu = None if step else _cu(0, 3, 3, 70)
    want, before = nv.conv_silu(x.contiguous(), w, cu_seqlens=cu), x.clone()
    nv.conv_silu(x, w, cu_seqlens=cu, out=y)
    assert torch.equal(y, want) and torch.equal(x, before)


@pytest.mark.parametrize("rows,cols", [(5, 5120), (70, 1033), (300, 100), (9, 15), (3, 16384), (1, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_in_place(rows, cols, dtype):
    print(f"[overlap] norms {rows}x{cols} {dtype}", flush=True)
    x, r, w = _rows(rows, cols, dtype, 1), _rows(rows, cols, dtype, 2), _rows(1, cols, F32, 3)[0]
    t = torch.empty_like(x)
    y = nv.add_rmsnorm(x, w, residual=r, scale=0.5, residual_out=t, out_dtype=dtype)
    for which in ("y on x", "y on r", "t on x", "t on r, y on x", "t on x, y on r"):
        a, b = x.clone(), r.clone()
        place = {p.split()[0]: a if p.endswith("x") else b for p in which.split(", ")}
        ty, tt = place.get("y", torch.empty_like(x)), place.get("t", torch.empty_like(x))
        nv.add_rmsnorm(a, w, residual=b, scale=0.5, residual_out=tt, out=ty)
        assert torch.equal(ty, y) and torch.equal(tt, t), which
    if cols % 16 == 0:
        wg = _rows(1, 16, F32, 4)[0]
        want = nv.rmsnorm_gated(x, r, wg, out_dtype=dtype)
        for on_z in (False, True):
            a, b = x.clone(), r.clone()
            nv.rmsnorm_gated(a, b, wg, out=b if on_z else a)
            assert torch.equal(b if on_z else a, want)


def test_refusals():
    dev = need_gpu()
    x, gates, lay = _tensors(8, 1, 2, 1)
    cu, st = _cu(0, 8), torch.zeros((8, 2, D, D), device=dev)
    pool = torch.zeros((9, 2, D, D), device=dev)
    n = _rows(9, 256, BF, 1)
    wn, wc = torch.ones(256, device=dev), torch.ones((256, 4), device=dev)
    gs, codes, scales = torch.ones(1, device=dev), n.view(torch.uint8).view(-1), torch.empty((8, 16), dtype=torch.uint8, device=dev)
    for bad in (lambda: nv.gdn_prefill(x, gates, cu, **lay, o=x), lambda: nv.gdn_prefill(x, gates, cu, **lay, o=x[:, 2 * D:]),
                lambda: nv.gdn_decode(x, gates, st, **lay, o=x), lambda: nv.gdn_decode(x, gates, st, **lay, o=x[:, D:]),
                lambda: nv.gdn_prefill(x, gates, cu, **lay, state_in=pool[:8], state_out=pool[1:]),
                lambda: nv.conv_silu(n, wc, out=n), lambda: nv.conv_silu(n[:8], wc, out=n[1:]),
                lambda: nv.add_rmsnorm(n[:8], wn, out=n[1:]), lambda: nv.add_rmsnorm(n[1:], wn, residual=n[:8], residual_out=n[1:], out=n[:8]),
                lambda: nv.add_rmsnorm(n, wn, residual=n, residual_out=n, out=n),
                lambda: nv.add_rmsnorm(n[:8], wn, y_gs=gs, codes=codes[:8 * 128].view(8, 128), scales=scales),
                lambda: nv.rmsnorm_gated(n[:8], n[1:], wn[:128], out=n[:8])):
        with pytest.raises(nv.Nvfp4Error, match="ALIAS"):
            bad()
