"""Rows past what one dimension of a grid holds: nvfp4_conv_silu takes up to
2^31 - 1 of them."""
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_rows_than_a_grid_dimension(dtype):
    """Windows of the long call's rows, at its ends, around sequences' starts and around multiples of 2^26 rows, have
    the bits of a call on them alone; every row is written."""
    dev = need_gpu()
    T, C = (1 << 28) + 37, 1
    print(f"[conv] {T} rows {dtype}", flush=True)
    x = torch.randn((T, C), generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(dtype)
    w = torch.randn((C, 4), generator=torch.Generator(device=dev).manual_seed(2), device=dev)
    starts = [0, 5, (1 << 27) + 3, T - 70]
    cu = torch.tensor([*starts, T], dtype=torch.int32, device=dev)
    y = torch.full((T, C), float("nan"), dtype=dtype, device=dev)
    state = torch.zeros((4, 3, C), dtype=dtype, device=dev)
    nv.conv_silu(x, w, cu_seqlens=cu, out=y, state=state)
    assert not bool(torch.isnan(y).any()), "rows were left out"
    for s in starts:
        assert torch.equal(y[s:s + 70], nv.conv_silu(x[s:s + 70].contiguous(), w, cu_seqlens=cu.new_tensor([0, 5, 70] if s == 0 else [0, 70])))
    for r in [*range(1 << 26, T, 1 << 26), T - 100]:
        want = nv.conv_silu(x[r - 103:r + 97].contiguous(), w, cu_seqlens=cu.new_tensor([0, 200 if r < T - 100 else 133, 200])[:3])
        n = 100 if r < T - 100 else 30
        assert torch.equal(y[r - 100:r - 100 + n], want[3:3 + n])
    for i, e in enumerate(starts[1:] + [T]):
        assert torch.equal(state[i], x[e - 3:e])
