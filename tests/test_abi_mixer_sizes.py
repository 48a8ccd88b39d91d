"""Largest sizes of the GDN mixer's calls, without a GPU.  A call that passes the
checks of sizes is told from one that does not by its missing pointers."""
import pytest

from nvfp4_w4a4_quantized_05_amd import _lib

NULL, SHAPE = 1, 2


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.mark.parametrize("rows,cols,want", [
    (1 << 22, 15360, NULL), (1 << 22, 15361, SHAPE), (1 << 22, 16384, SHAPE), ((1 << 22) - 1, 16384, NULL), (1 << 22, 1, NULL)])
def test_add_rmsnorm_keeps_its_grid_below_2_to_32_threads(lib, rows, cols, want):
    """More would be cut to 32 bits by the launch, without an error."""
    assert lib.nvfp4_add_rmsnorm(None, 1, cols, None, 1, 0, 1.0, None, 1e-6, rows, cols, None, 0, None, 1, cols, None, None,
                                 None, None) == want


@pytest.mark.parametrize("cols", [16, 48, 80, 4096, 5120])
def test_rmsnorm_gated_takes_less_than_2_to_35_values(lib, cols):
    most = ((1 << 35) - 1) // cols
    for rows, want in ((most, NULL), (most + 1, SHAPE)):
        assert lib.nvfp4_rmsnorm_gated(None, 1, cols, None, 1, cols, None, 1e-6, rows, cols, 16, None, 1, cols, None, None, None,
                                       None) == want
