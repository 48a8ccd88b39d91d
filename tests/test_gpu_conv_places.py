"""nvfp4_conv_silu with a sequence that starts at every place of a tile of 16
rows, for every width; checks and allowance as in test_gpu_conv.py."""
import pytest
import torch

from tests.test_gpu_conv import BF, F32, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("place", range(16))
@pytest.mark.parametrize("width", [2, 3, 4])
def test_start(place, width):
    n = 48 + place
    _case([n, 1, 1, 2, 40], 16, width, BF, place)
    _case([n, 2, 30], 24, width, F32, place, skip=(1,))
    _case([n, 17, 0, 3], 9, width, BF, place, pool=False, tail=1)
    _case([n, 3, 15], 5, width, F32, place, skip=(0, 2), pad=1)
