"""One token, or one row, whose tensors have a number of columns that is no
multiple of 8 (q, k, v and the gates in one row): a single row's stride is no
address, so such a call is the same as the first row of a longer one."""
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import need_gpu
from tests.test_gpu_gdn_serve import BF, D, F32, _cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_qk,n_v,more", [(1, 3, 0), (2, 2, 1), (1, 1, 5)])
def test_one_row_of_the_whole_projection(dtype, n_qk, n_v, more):
    dev = need_gpu()
    w = D * (2 * n_qk + n_v)
    cols = w + 2 * n_v + more                         # q | k | v | g | beta | other columns
    print(f"[one row] heads {n_qk}/{n_v}, {cols} columns, {dtype}", flush=True)
    buf = torch.randn((2, -(-cols // 8) * 8), generator=torch.Generator(device=dev).manual_seed(cols), device=dev).to(dtype)
    buf[:, w:w + n_v] = -buf[:, w:w + n_v].abs()
    lay = dict(q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=w, beta_col=w + n_v, n_qk_heads=n_qk, n_v_heads=n_v)
    rows, one = buf[:, :cols], buf[:1, :cols]
    st = [torch.zeros((2, n_v, D, D), device=dev) for _ in range(2)]
    o = [torch.zeros((n, -(-cols // 8) * 8), dtype=dtype, device=dev)[:, :cols] for n in (2, 1)]
    for x, s, out in ((rows, st[0], o[0]), (one, st[1], o[1])):
        nv.gdn_decode(x, x, s, **lay, o=out)
    assert torch.equal(o[1][0], o[0][0]) and torch.equal(st[1][0], st[0][0])
    if dtype == BF:
        for x, out, cu in ((rows, o[0], _cu(0, 1, 2)), (one, o[1], _cu(0, 1))):
            nv.gdn_prefill(x, x, cu, **lay, o=out)
        assert torch.equal(o[1][0], o[0][0])
        assert nv.gdn_prefill(one[:0], one[:0], _cu(0, 0), **lay, o=o[1][:0]).shape == (0, cols)
