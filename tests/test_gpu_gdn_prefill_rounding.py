"""nvfp4_gdn_prefill's o is the fp64 result rounded once to bf16, as near as
operands of two bf16 terms come to it.

Allowance, with the names of test_gpu_gdn_serve.py: before its rounding o is off
by the state's error e_t and by the fp32 sums, 400 u M_t; the chunk's start state
enters with 16 bits or more (2^-15 of it: the first term rounded, 2^-8, the second
cut off, 2^-7 of the rest), the scores and the writes rounded to 16 bits (2^-16
each) without the product of their second terms (2^-16 of the product):
|d_t| <= [e_t + 2^-15 |S_{s-1}|_F a_t + 3 2^-16 sum_j a_{t,j} |qhat_t . khat_j| |w_j|
+ 400 u M_t] / sqrt(128) as a vector.  Rounding then adds half a bf16 ulp of each
value: 2^(e - 8) for a value of exponent e.  What an error is larger than that half
ulp must be a vector no longer than d_t."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import host_f32, need_gpu
from tests.test_gpu_gdn_serve import BF, D, F32, U, _bounds, _host, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [True, False])
@pytest.mark.parametrize("many,n_qk,n_v", [(1, 2, 4), (50, 1, 4), (70, 1, 8)])  # 12, 208 and 568 sequences x heads
@pytest.mark.parametrize("decay", [3.0, 0.3, 0.01])
def test_outputs_are_rounded_once(many, n_qk, n_v, decay, start):
    """From a zero state the first tokens' outputs are scores times writes alone."""
    dev = need_gpu()
    lens = [150, 64, 9] + [3] * (many - 1)
    print(f"[rounding] {len(lens)} sequences, heads {n_qk}/{n_v}, decay {decay}, start {start}", flush=True)
    T, n = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, g, beta = _inputs(T, n_qk, n_v, int(100 * decay) + many)
    g = (-decay * np.random.default_rng(many).uniform(0.5, 1.5, g.shape)).astype(np.float32)
    pool = torch.randn((n, n_v, D, D), generator=torch.Generator().manual_seed(many)) * 0.3
    o = nv.gdn_prefill(torch.from_numpy(x).to(dev).to(BF), torch.from_numpy(np.concatenate([g, beta], 1)).to(dev),
                       torch.from_numpy(cu).to(dev), q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v,
                       n_qk_heads=n_qk, n_v_heads=n_v, state_in=pool.to(dev) if start else None)
    torch.cuda.synchronize()
    q, k, v, g, beta = _host(x, g, beta, n_qk, n_v)
    O, _, e, Mt, half, _, _ = _bounds(q, k, v, g, beta, cu, list(pool.numpy()) if start else None, 400)
    # half = 2^-9 |S| a + 2^-8 sum: 2^-6 of it is 2^-15 |S| a + 2^-14 sum
    d = (e + 2.0 ** -6 * half + 400 * U * Mt) / np.sqrt(D)
    got = host_f32(o).astype(np.float64).reshape(O.shape)
    ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(O) + d[..., None], 2.0 ** -126))) - 8)
    over = np.linalg.norm(np.maximum(np.abs(got - O) - ulp, 0), axis=2)
    print(f"  worst excess / allowance {np.max(over / d):.3f}", flush=True)
    assert np.all(over <= d), f"{np.count_nonzero(over > d)} rows, worst {np.max(over / d)}"
