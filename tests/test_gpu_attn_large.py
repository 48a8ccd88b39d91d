"""nvfp4_attn_cached with scores far outside what a softmax meets in earnest: finite queries and keys give finite
rows, and weights go by the scores' differences.  Bounds: tests/test_host_attn.py."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv
from tests.attn_util import Paged, i32
from tests.gpu_util import host_f32, need_gpu
from tests.test_gpu_attn import run
from tests.test_host_attn import FACTORS, FACTORS_OF_SCORES, check_common_part, check_one_hot, common_part

pytestmark = pytest.mark.gpu

# heads, head size, page; rows of each sequence, what each has before them: 16, 32 and 128 rows at a time, then with a
# range for every wave
SHAPES = [((4, 2, 128, 16), [1, 2], [1290, 2]), ((6, 1, 256, 32), [5, 4], [600, 1]), ((4, 1, 64, 16), [20, 30], [460, 0]),
          ((6, 1, 256, 64), [40, 25], [400, 3]), ((8, 8, 64, 16), [1] * 72, [90] * 71 + [1500]),
          ((8, 8, 128, 16), [20] * 18, [40] * 17 + [900])]


def call(paged, q, rows, kv, hq, scale):
    dev = need_gpu()
    cache, table = paged.to(dev)
    starts = np.concatenate([[0], np.cumsum(rows)])
    o = nv.attn_cached(q, cache, table, i32(kv, dev), i32(starts, dev), n_q_heads=hq, scale=scale)
    return host_f32(o), starts


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("factor", FACTORS)
def test_finite_queries_of_any_size(fmt, shape, factor):
    (hq, hk, d, page), rows, ctx = SHAPES[shape]
    kv = [a + b for a, b in zip(rows, ctx)]
    print(f"[attn] {fmt} shape {shape} queries of {factor}", flush=True)
    paged = Paged(fmt, hk, d, page, kv, 21)
    g = np.random.default_rng(5)
    q = torch.from_numpy((factor * g.standard_normal((sum(rows), hq * d))).astype(np.float32)).to(need_gpu()).bfloat16()
    got, starts = call(paged, q, rows, kv, hq, None)
    check_one_hot(got, host_f32(q).astype(np.float64), paged, kv, rows, starts, hq, float(np.float32(d ** -0.5)))


@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_large_scores_that_differ_little(shape):
    (hq, hk, d, page), rows, ctx = SHAPES[shape]
    kv = [a + b for a, b in zip(rows, ctx)]
    print(f"[attn] shape {shape} large scores", flush=True)
    paged, q, scale = common_part(hk, d, page, kv, hq // hk, sum(rows), 22)
    got, starts = call(paged, torch.from_numpy(q).to(need_gpu()).bfloat16(), rows, kv, hq, scale)
    check_common_part(got, q, paged, rows, kv, starts, hq, scale)


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("scale,k_gs,spread", FACTORS_OF_SCORES)
def test_factors_whose_product_is_no_fp32_number(shape, scale, k_gs, spread):
    (hq, hk, d, page), rows, ctx = SHAPES[shape]
    kv = [a + b for a, b in zip(rows, ctx)]
    print(f"[attn] shape {shape} scale {scale} {k_gs}", flush=True)
    run(Paged("fp8", hk, d, page, kv, 23, k_gs=k_gs), rows, kv, hq, scale=scale, spread=spread)
