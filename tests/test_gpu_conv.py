"""nvfp4_conv_silu against the fp64 formula.

Tolerance: the fp32 sum of `width` fused products is off by at most width u
sum |w x| =: width u m (u = 2^-24); silu has a slope of at most 1.1, and its own
exp2 argument, exp2, sum, reciprocal and product give (2 |s| + 5) u of the
result: |y - Y| <= u (1.1 width m + (2 |s| + 5) |Y|), plus half a bf16 ulp (2^-8)
for bf16.  The states are copies and must be equal."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from oracle import mixer_ref as M
from tests.gpu_util import host_f32, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _case(lens, channels, width, dtype, seed, *, step=False, pool=True, pad=0, skip=(), tail=0):
    """Runs one call and checks y, the slots it owns, and what it must not touch."""
    dev = need_gpu()
    print(f"[conv] lens {lens if len(lens) < 12 else len(lens)} C {channels} W {width} {dtype} step {step}", flush=True)
    rng = np.random.default_rng(seed)
    n, T = len(lens), sum(lens) + tail
    cu = np.concatenate([[0], np.cumsum(lens)])
    buf = torch.full((T, channels + pad), float("nan"), dtype=dtype, device=dev)
    buf[:sum(lens), :channels] = torch.from_numpy(rng.standard_normal((sum(lens), channels)).astype(np.float32)).to(dev).to(dtype)
    x = buf[:, :channels]
    w = torch.from_numpy(rng.standard_normal((channels, width)).astype(np.float32)).to(dev)
    slots = rng.permutation(n + 3)[:n].astype(np.int32)
    for i in skip:
        slots[i] = -1 if i % 2 else n + 3
    state = torch.from_numpy(rng.standard_normal((n + 3, width - 1, channels)).astype(np.float32)).to(dev).to(dtype)
    before = state.clone()
    y = torch.full((T, channels + pad), float("nan"), dtype=dtype, device=dev)
    nv.conv_silu(x, w, cu_seqlens=None if step else torch.from_numpy(cu.astype(np.int32)).to(dev),
                 state=state if pool else None, slots=torch.from_numpy(slots).to(dev) if pool else None, out=y)
    torch.cuda.synchronize()
    live = [i for i in range(n) if i not in skip]
    old = np.zeros((n, width - 1, channels), np.float32)
    if pool:
        old[live] = host_f32(before)[slots[live]]
    Y, mag, new = M.conv_silu_ref(np.nan_to_num(host_f32(x)), w.cpu().numpy(), cu, old)
    got = host_f32(y).astype(np.float64)
    s = mag                                       # |s| <= the magnitude sum
    tol = U * (1.1 * width * mag + (2 * s + 5) * np.abs(Y)) + 2.0 ** -120
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(Y) + tol)
    for i in range(n):
        a, b = cu[i], cu[i + 1]
        if i in skip:
            assert np.all(got[a:b, :channels] == 0), f"sequence {i} is skipped: zeros"
            continue
        err = np.abs(got[a:b, :channels] - Y[a:b])
        assert np.all(err <= tol[a:b]), f"sequence {i}: worst error / tolerance {np.max(err / tol[a:b])}"
    assert np.all(np.isnan(got[sum(lens):])), "rows of no sequence were written"
    if pad:
        assert np.all(np.isnan(got[:, channels:])), "columns past the channels were written"
    if pool:
        want = host_f32(before).copy()
        want[slots[live]] = new[live]
        assert np.array_equal(host_f32(state), want), "state pool"


@pytest.mark.parametrize("lens,channels,width,dtype", [
    ([1], 8, 4, BF), ([2], 16, 4, F32), ([3], 8, 4, BF), ([200], 256, 4, BF), ([64], 64, 3, F32), ([65], 64, 2, BF),
    ([63, 1, 64, 2, 70], 2056, 4, BF), ([0, 1, 0, 2, 3, 0, 130, 1, 1], 136, 4, F32), ([1] * 70, 40, 4, BF),
    ([61, 5, 1, 61, 3], 8, 3, BF)])
def test_packed(lens, channels, width, dtype):
    _case(lens, channels, width, dtype, len(lens) * 100 + channels)
    _case(lens, channels, width, dtype, len(lens) * 100 + channels, pool=False, tail=3)


@pytest.mark.parametrize("lens,channels,width,dtype,pad", [
    ([1, 5], 1, 4, BF, 0), ([70, 0, 3], 13, 4, F32, 0), ([129], 321, 3, BF, 1), ([30], 64, 2, F32, 1),
    ([64, 64], 256, 4, BF, 8)])
def test_packed_odd_channels_and_strides(lens, channels, width, dtype, pad):
    _case(lens, channels, width, dtype, channels, pad=pad, tail=2)


@pytest.mark.parametrize("starts", range(58, 71))
def test_a_sequence_that_starts_at_every_place_of_a_tile(starts):
    _case([starts, 1, 1, 2, 90], 16, 4, BF, starts)
    _case([starts, 80], 16, 4, F32, starts, skip=(1,))


@pytest.mark.parametrize("batch,channels,width,dtype,pad", [
    (1, 8192, 4, BF, 0), (64, 2056, 4, BF, 0), (5, 13, 3, F32, 2), (9, 64, 2, F32, 0), (130, 8, 4, BF, 8)])
def test_step(batch, channels, width, dtype, pad):
    _case([1] * batch, channels, width, dtype, batch, step=True, pad=pad, skip=(2, 3) if batch > 4 else ())
    _case([1] * batch, channels, width, dtype, batch, step=True, pool=False)


def test_skipped_sequences():
    _case([5, 70, 0, 3, 64, 1], 24, 4, BF, 3, skip=(0, 1, 3, 5))


def test_steps_after_a_prompt_equal_the_whole_prompt():
    """Packed in one call, in two calls, and token by token: the same bits."""
    dev = need_gpu()
    x = torch.randn((90, 520), device=dev).to(BF)
    w = torch.randn((520, 4), device=dev)
    cu = lambda *c: torch.tensor(c, dtype=torch.int32, device=dev)
    st = torch.zeros((1, 3, 520), dtype=BF, device=dev)
    want = nv.conv_silu(x, w, cu_seqlens=cu(0, 90), state=st)
    end = st.clone()
    st.zero_()
    a = nv.conv_silu(x[:2], w, cu_seqlens=cu(0, 2), state=st)
    b = nv.conv_silu(x[2:80], w, cu_seqlens=cu(0, 78), state=st)
    rest = [nv.conv_silu(x[t:t + 1], w, state=st) for t in range(80, 90)]
    assert torch.equal(torch.cat([a, b, *rest]), want) and torch.equal(st, end)


def test_a_bad_request_does_not_reach_its_neighbours():
    dev = need_gpu()
    x = torch.randn((30, 64), device=dev).to(BF)
    w = torch.randn((64, 4), device=dev)
    cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device=dev)
    want = nv.conv_silu(x, w, cu_seqlens=cu)
    x[10:20] = float("nan")
    got = nv.conv_silu(x, w, cu_seqlens=cu)
    keep = list(range(10)) + list(range(20, 30))
    assert torch.equal(got[keep], want[keep])


def test_refusals():
    dev = need_gpu()
    x = torch.zeros((4, 64), dtype=BF, device=dev)
    w = torch.zeros((64, 4), device=dev)
    st = torch.zeros((2, 3, 64), dtype=BF, device=dev)
    sl = torch.zeros(4, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    for bad in (lambda: nv.conv_silu(x, w.to(BF)), lambda: nv.conv_silu(x, w[:32]), lambda: nv.conv_silu(x.half(), w),
                lambda: nv.conv_silu(x, w, state=st.float()), lambda: nv.conv_silu(x, w, state=st[:, :2]),
                lambda: nv.conv_silu(x, w, slots=sl), lambda: nv.conv_silu(x, w, state=st, slots=sl[:3]),
                lambda: nv.conv_silu(x, w, cu_seqlens=cu.long()), lambda: nv.conv_silu(x, w, cu_seqlens=cu[:1]),
                lambda: nv.conv_silu(x, w, out=x[:2]), lambda: nv.conv_silu(x.cpu(), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.conv_silu(x, w, out=x), lambda: nv.conv_silu(x, torch.zeros((64, 5), device=dev)),
                lambda: nv.conv_silu(x, torch.zeros((64, 1), device=dev))):
        with pytest.raises(nv.Nvfp4Error):
            bad()
    assert nv.conv_silu(x[:0], w).shape == (0, 64)


@pytest.mark.parametrize("channels,dtype", [(7, BF), (9, BF), (2049, BF), (2055, BF), (3, F32), (5, F32), (1025, F32), (1027, F32)])
def test_channels_that_end_inside_a_vector(channels, dtype):
    """The last lane takes channels that the lane before it has too: in the same wave, or in another workgroup."""
    _case([40, 1, 2, 0, 3, 17], channels, 4, dtype, channels, pad=1, tail=1)
    _case([1] * 9, channels, 4, dtype, channels, step=True, pad=1, skip=(4,))
