"""Sums beyond the 16-bit type's range: z_out then holds an infinity while the output, from the FP32 sum, is finite, and
the backward pass at that z has the activation's limit slopes, 0 and 1."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_fp16_sums_below_the_range_have_no_gradient(act):
    M, K, N = 3, 8, 16
    x = torch.ones((M, K), dtype=torch.float16, device="cuda")
    w = torch.zeros((N, K), dtype=torch.float16, device="cuda")
    w[1] = 1.0
    bias = torch.zeros(N, device="cuda")
    bias[0] = -1e5                                             # z = -1e5 in FP32, -inf in FP16
    y, z = moe.linear(x, w, bias=bias, act=act, save_z=True)
    assert (z[:, 0] == -torch.inf).all() and torch.isfinite(y).all() and (y[:, 0] == 0).all()
    dy = torch.full((M, N), 2.0, dtype=torch.float16, device="cuda")
    dx, dw, db = moe.linear_backward(dy, x, w, z=z, act=act, bias=True)
    assert all(torch.isfinite(t).all() for t in (dx, dw, db))
    assert (dw[0] == 0).all() and db[0] == 0
    # as if the column were not there
    dy0 = dy.clone()
    dy0[:, 0] = 0
    z0 = z.clone()
    z0[:, 0] = 0
    for a, b in zip((dx, dw, db), moe.linear_backward(dy0, x, w, z=z0, act=act, bias=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_slopes_at_infinity(act, dtype):
    z = torch.zeros((1, 8), dtype=dtype, device="cuda")
    z[0, 0], z[0, 1], z[0, 2] = -torch.inf, torch.inf, torch.nan
    big = torch.finfo(dtype).max
    z[0, 3], z[0, 4] = -big, big
    dy = torch.full((1, 8), -3.0, dtype=dtype, device="cuda")
    w = torch.eye(8, dtype=dtype, device="cuda")
    dx, _, db = moe.linear_backward(dy, w[:1].contiguous(), w, z=z, act=act, bias=True)
    want = [-3.0, -3.0] if act == "none" else [0.0, -3.0]
    np.testing.assert_array_equal(db[[0, 1]].double().cpu().numpy(), want)
    np.testing.assert_array_equal(db[[3, 4]].double().cpu().numpy(), want)
    assert act == "none" or torch.isnan(db[2])
    assert torch.isnan(dx).all() if act != "none" else (dx == -3).all()          # the NaN passes w's zeros
