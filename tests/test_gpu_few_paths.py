"""moe_forward_few on the GPU: paths and reports that the cases of
test_gpu_few.py do not reach."""
from __future__ import annotations

import pytest
import torch

from mixture_experts_layer_41_b200 import _lib as L
from mixture_experts_layer_41_b200 import api
from test_gpu_few import few, make_run

pytestmark = pytest.mark.gpu


def test_few_wait_limit_names_its_kernel():
    """A grid barrier that runs out is reported as the few-token kernel's, not as
    a tensor-core kernel's."""
    run = make_run("long_rows")
    try:
        api.moe_set_wait_timeout_ns(1)
        few(run)
        assert run.status() == L.MOE_ERR_DEVICE
        text = L.lib().moe_last_error().decode()
    finally:
        api.moe_set_wait_timeout_ns(0)
    assert "few-token kernel" in text and "timed out" in text and "tensor-core" not in text, text
    few(run)
    torch.cuda.synchronize()
    assert run.status() == 0
