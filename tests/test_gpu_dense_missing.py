"""Gradients of the products without the operands they do not need: the bits of the full calls."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


@pytest.mark.parametrize("rows", [0, 1, 90, 2000])
def test_missing_operands(rows):
    x, w = torch.randn((rows, 136), device="cuda").bfloat16(), torch.randn((3, 72, 136), device="cuda").bfloat16()
    dy = torch.randn((rows, 72), device="cuda").bfloat16()
    o = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    dx, dw = moe.grouped_mm_backward(dy, x, w, o)
    assert torch.equal(moe.grouped_mm_backward(dy, x, None, o, need_dx=False)[1], dw)
    assert torch.equal(moe.grouped_mm_backward(dy, None, w, o, need_dw=False)[0], dx)
    dx, dw, db = moe.linear_backward(dy, x, w[0], z=dy, act="gelu", bias=True)
    none, dw1, db1 = moe.linear_backward(dy, x, None, z=dy, act="gelu", bias=True, need_dx=False)
    assert none is None and torch.equal(dw1, dw) and torch.equal(db1, db)
    dx2, none, db2 = moe.linear_backward(dy, None, w[0], z=dy, act="gelu", bias=True, need_dw=False)
    assert none is None and torch.equal(dx2, dx) and torch.equal(db2, db)
    n1, n2, db3 = moe.linear_backward(dy, None, None, z=dy, act="gelu", bias=True, need_dx=False, need_dw=False)
    assert n1 is None and n2 is None and torch.equal(db3, db)
