"""Finite q and k whose squared length is past fp32's range, in prefill and
decode: khat and qhat are unit vectors as for any other row.  Allowances as in
test_gpu_gdn_serve.py (a row that is multiplied by a power of two loses no bits
but of values 2^-100 of its largest)."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.gpu_util import host_f32, need_gpu
from tests.test_gpu_gdn_serve import BF, D, F32, U, _bounds, _host, _inputs

pytestmark = pytest.mark.gpu


def _large(T, n_qk, n_v, seed, part, size):
    """_inputs with some rows' q or k (or both) of about `size`; one of them with a single large value."""
    x, g, beta = _inputs(T, n_qk, n_v, seed)
    rng = np.random.default_rng(seed + 1)
    with np.errstate(over="ignore"):
        for which, at in (("q", 0), ("k", n_qk * D)):
            if which in part:
                rows = rng.random(T) < 0.4
                rows[0] = True
                block = x[:, at:at + n_qk * D]
                block[rows] = np.clip(block[rows].astype(np.float64) / 4 * size, -3.3e38, 3.3e38)
                one = int(rng.integers(0, T))
                block[one] = rng.standard_normal(n_qk * D)
                block[one, ::D] = size
    x = torch.from_numpy(x).to(BF).float().numpy()
    assert np.all(np.isfinite(x))
    return x, g, beta


SIZES = [4e15, 2e18, 3e19, 1e30, 3e38]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("part,many", [("k", 1), ("q", 1), ("qk", 1), ("qk", 50), ("qk", 130)])
def test_prefill(part, many, size):
    dev = need_gpu()
    n_qk, n_v = 2, 4
    lens = [150, 70] + [2] * (many - 1)
    print(f"[large] prefill {part} {size:g}, {len(lens)} sequences", flush=True)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, g, beta = _large(sum(lens), n_qk, n_v, many, part, size)
    pool = torch.randn((len(lens), n_v, D, D), generator=torch.Generator().manual_seed(1)) * 0.3
    state = pool.to(dev)
    o = nv.gdn_prefill(torch.from_numpy(x).to(dev).to(BF), torch.from_numpy(np.concatenate([g, beta], 1)).to(dev),
                       torch.from_numpy(cu).to(dev), q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v,
                       n_qk_heads=n_qk, n_v_heads=n_v, state_in=state, state_out=state)
    torch.cuda.synchronize()
    q, k, v, g, beta = _host(x, g, beta, n_qk, n_v)
    O, S, e, Mt, half, _, final = _bounds(q, k, v, g, beta, cu, list(pool.numpy()), 400)
    tol = (e + half + 400 * U * Mt) / np.sqrt(D) + 2.0 ** -8 * np.linalg.norm(O, axis=2)
    err = np.linalg.norm(host_f32(o).astype(np.float64).reshape(O.shape) - O, axis=2)
    assert np.all(err <= tol), f"{np.count_nonzero(~(err <= tol))} rows, worst {np.nanmax(err / tol)}"
    es = np.linalg.norm((state.cpu().numpy() - S).reshape(len(lens), n_v, -1), axis=2)
    assert np.all(es <= final), f"state, worst {np.nanmax(es / final)}"


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("part,batch,n_qk,n_v", [("k", 6, 2, 4), ("q", 6, 2, 4), ("qk", 40, 8, 32)])
def test_decode(part, batch, n_qk, n_v, dtype, size):
    dev = need_gpu()
    print(f"[large] decode {part} {size:g}, {batch} x {n_v} heads {dtype}", flush=True)
    x, g, beta = _large(batch, n_qk, n_v, batch, part, size)
    pool = torch.randn((batch, n_v, D, D), generator=torch.Generator().manual_seed(1)) * 0.3
    state = pool.to(dev)
    o = nv.gdn_decode(torch.from_numpy(x).to(dev).to(dtype), torch.from_numpy(np.concatenate([g, beta], 1)).to(dev), state,
                      q_col=0, k_col=n_qk * D, v_col=2 * n_qk * D, g_col=0, beta_col=n_v, n_qk_heads=n_qk, n_v_heads=n_v,
                      o=torch.empty((batch, n_v * D), device=dev))
    torch.cuda.synchronize()
    q, k, v, g, beta = _host(x, g, beta, n_qk, n_v)
    O, S, e, Mt, _, _, _ = _bounds(q, k, v, g, beta, np.arange(batch + 1), list(pool.numpy()), 160)
    err = np.linalg.norm(o.double().cpu().numpy().reshape(O.shape) - O, axis=2)
    tol = 4 * 144 * U * Mt / np.sqrt(D)
    assert np.all(err <= tol), f"o, worst {np.nanmax(err / tol)}"
    es = np.linalg.norm((state.cpu().numpy() - S).reshape(batch, n_v, -1), axis=2)
    assert np.all(es <= e), f"state, worst {np.nanmax(es / e)}"
