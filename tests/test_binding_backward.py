"""The binding of the products' backward calls without the operands a gradient does not need: checked here up to the
device check, which names the first tensor that is not on a GPU."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

X, W, DY = torch.zeros((6, 64)).bfloat16(), torch.zeros((4, 32, 64)).bfloat16(), torch.zeros((6, 32)).bfloat16()
OFF = torch.zeros(5, dtype=torch.int32)


def test_operands_that_are_not_needed_may_be_missing():
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        moe.grouped_mm_backward(DY, X, None, OFF, need_dx=False)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        moe.grouped_mm_backward(DY, None, W, OFF, need_dw=False)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        moe.linear_backward(DY, X, None, need_dx=False)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        moe.linear_backward(DY, None, W[0], need_dw=False)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        moe.linear_backward(DY, None, None, bias=True, need_dx=False, need_dw=False)


def test_operands_that_are_needed():
    for f, a in ((moe.grouped_mm_backward, (OFF,)), (moe.linear_backward, ())):
        w = W if a else W[0]
        with pytest.raises(ValueError, match="dx needs w"):
            f(DY, X, None, *a)
        with pytest.raises(ValueError, match="dx needs w"):
            f(DY, X, None, *a, need_dx=False, dx=torch.zeros((6, 64)).bfloat16())
        with pytest.raises(ValueError, match="dw needs x"):
            f(DY, None, w, *a)
        with pytest.raises(ValueError, match="dw needs x"):
            f(DY, None, w, *a, need_dw=False, dw=torch.zeros_like(w))


def test_shapes_without_w():
    f = moe.grouped_mm_backward
    with pytest.raises(TypeError, match="offsets must be a 1-D tensor"):
        f(DY, X, None, OFF[None], need_dx=False)
    with pytest.raises(TypeError, match=r"x must have shape \(6, 64\)"):
        f(DY, X[:5], None, OFF, need_dx=False)
    with pytest.raises(TypeError, match=r"dw must have shape \(4, 32, 64\)"):
        f(DY, X, None, OFF, need_dx=False, dw=torch.zeros((5, 32, 64)).bfloat16())
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        f(DY, X.half(), None, OFF, need_dx=False)
    with pytest.raises(TypeError, match="x must be a 2-D tensor"):
        moe.linear_backward(DY, X[0], None, need_dx=False)
    with pytest.raises(TypeError, match=r"dw must have shape \(32, 64\)"):
        moe.linear_backward(DY, X, None, need_dx=False, dw=torch.zeros((32, 56)).bfloat16())
