"""Packed calls whose cu_seqlens hold row numbers outside 0 .. T: the same bits,
in outputs and slots, as with the numbers cut off there."""
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import need_gpu
from tests.test_gpu_gdn_serve import BF, D, F32, _tensors

pytestmark = pytest.mark.gpu

# row numbers, rows
CASES = [([-3, 40], 40), ([-1, 0, 40], 40), ([-70, -2, 33, 90], 90), ([-5, 100, 1000], 100), ([0, 7, 50, 51, 64], 50),
         ([-2 ** 31, 17, 2 ** 31 - 1], 130), ([-9, -4, -1], 20), ([60, 70, 80], 60), ([-20, 1, 2, 500], 33)]


def _both(cu, T, call):
    """call(cu_seqlens) for the numbers as they are and cut off."""
    dev = need_gpu()
    return [call(torch.tensor(c, dtype=torch.int32, device=dev)) for c in (cu, [min(max(x, 0), T) for x in cu])]


@pytest.mark.parametrize("cu,T", CASES)
@pytest.mark.parametrize("channels,dtype", [(136, BF), (13, F32)])
def test_conv(cu, T, channels, dtype):
    dev = need_gpu()
    print(f"[conv rows] {cu} of {T}, {channels} channels", flush=True)
    g = torch.Generator(device=dev).manual_seed(T)
    x = torch.randn((T, channels), generator=g, device=dev).to(dtype)
    w = torch.randn((channels, 4), generator=g, device=dev)
    pool = torch.randn((len(cu), 3, channels), generator=g, device=dev).to(dtype)

    def call(c):
        state, y = pool.clone(), torch.full_like(x, 7.0)
        nv.conv_silu(x, w, cu_seqlens=c, state=state, out=y)
        return y, state

    (y, state), (want, want_state) = _both(cu, T, call)
    assert torch.equal(y, want) and torch.equal(state, want_state)


@pytest.mark.parametrize("cu,T", CASES)
def test_prefill(cu, T):
    print(f"[prefill rows] {cu} of {T}", flush=True)
    x, gates, lay = _tensors(T, 1, 2, T)
    pool = torch.randn((len(cu), 2, D, D), generator=torch.Generator(device=x.device).manual_seed(T), device=x.device)

    def call(c):
        state, o = pool.clone(), torch.full((T, 2 * D), 7.0, dtype=BF, device=x.device)
        nv.gdn_prefill(x, gates, c, **lay, state_in=state, state_out=state, o=o)
        return o, state

    (o, state), (want, want_state) = _both(cu, T, call)
    assert torch.equal(o, want) and torch.equal(state, want_state)
