"""Single gradients of a batch without rows: torch hands out a null pointer for an output without elements."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu


def test_dx_alone_without_rows():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    x, dy = (torch.empty((0, n), dtype=torch.bfloat16, device="cuda") for n in (24, 16))
    w, o = torch.ones((3, 16, 24), device="cuda").bfloat16(), torch.zeros(4, dtype=torch.int32, device="cuda")
    dx, dw = moe.grouped_mm_backward(dy, x, w, o, need_dw=False)
    assert dx.shape == (0, 24) and dw is None and moe.last_device_status() == moe.OK
    dx, dw, db = moe.linear_backward(dy, x, w[0], z=dy, act="silu", need_dw=False)
    assert dx.shape == (0, 24) and dw is None and db is None and moe.last_device_status() == moe.OK
    dx, dg, db = moe.layer_norm_backward(dy, dy, None, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 16) and dg is None and db is None
