"""What the attention layer's binding refuses before it calls the library: checked on host tensors that pass for the GPU's."""
import pytest
import torch

import nvfp4_w4a4_quantized_05_amd as nv


class Fake(torch.Tensor):
    is_cuda = True


def fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Fake)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("cols,kw", [(512, dict(q_col=0, k_col=512)), (760, dict(q_col=0, k_col=512)), (764, dict(q_col=0, k_col=512)),
                                     (768, dict(q_col=264, k_col=0)), (768, dict(q_col=0, k_col=520)), (768, dict(q_col=-8, k_col=512))])
def test_heads_outside_the_columns_of_x(T, cols, kw):
    """A view of fewer columns than its rows are apart: the heads must lie in what was given, not in the stride."""
    x = fake(T, 1024, dtype=torch.bfloat16)[:, :cols]
    with pytest.raises(ValueError, match="columns of x"):
        nv.qk_norm_rope(x, fake(128), fake(128), fake(4, 64), fake(T, dtype=torch.int32), n_q_heads=4, n_kv_heads=2, **kw)
