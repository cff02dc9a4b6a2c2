"""moe_quantized_matmul's weight shapes (no GPU)."""
import pytest
import torch

from mixture_experts_layer_41_b200 import api


@pytest.mark.parametrize("shape", [(2, 3, 32, 64), (1, 1, 32, 64), (64,)])
def test_matmul_refuses_weights_of_other_dimensions(shape, monkeypatch):
    """A stack of stacks would be taken for its first matrix."""
    monkeypatch.setattr(api, "_have_gpu", lambda: False)
    i8 = torch.int8
    with pytest.raises(ValueError, match="w_codes"):
        api.moe_quantized_matmul(torch.zeros((4, 64), dtype=i8), torch.zeros(4), torch.zeros(shape, dtype=i8), torch.zeros(32),
                                 torch.zeros((4, 32)), torch.zeros(256, dtype=torch.uint8), stream=0)
