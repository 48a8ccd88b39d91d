"""nvfp4_qk_norm_rope on heads whose squares are past fp32, up to the top of its range: tests/test_gpu_rope.py's check
and bound."""
import pytest
import torch

from tests.test_gpu_rope import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,adjacent", [(64, 32, False), (128, 128, True), (256, 64, False)])
@pytest.mark.parametrize("spread", [1e14, 1e16, 3e17, 2e18, 1e19, 1e25, 1e37, 6e37])
def test_squares_past_fp32(spread, d, rot, adjacent, dtype):
    run(21, 5, 2, d, rot, dtype, adjacent=adjacent, spread=spread)
