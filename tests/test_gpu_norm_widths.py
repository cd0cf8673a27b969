"""Layer norm at the widths where its kernels' shapes change: the last columns that one holds and the first of the next,
for rows of whole vectors and rows that start inside one, few rows and many."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_norm import E, check, f64

pytestmark = pytest.mark.gpu

HELD = [256, 1024, 2048, 4096, 5120, 6144, 8192, 16384]
WIDTHS = sorted({h + d for h in HELD for d in (-8, -7, -6, -4, -3, -1, 1, 8)} |
                {3064, 3065, 3066, 3068, 3069, 3071, 3073, 3080})


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [19, 333])
def test_widths_around_the_shapes(rows, dtype, cols):
    gen = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn((rows, cols), generator=gen) * 3 + 0.7).to(dtype)
    dy = torch.randn((rows, cols), generator=gen).to(dtype)
    gamma, beta = 1 + 0.2 * torch.randn(cols, generator=gen), torch.randn(cols, generator=gen)
    X, D, G, B = f64(x), f64(dy), f64(gamma), f64(beta)
    Y, MEAN, R = dense.layer_norm(X, G, B, float(np.float32(1e-2)))
    y, mean, rstd = moe.layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), eps=1e-2, stats=True)
    em = 48 * E * np.abs(X).mean(1) + E * np.abs(MEAN)
    er = R * (29 * E + 0.5 * (em * R) ** 2)
    rel = (er / R)[:, None] + 8 * E
    check(mean, MEAN, em, "mean")
    check(rstd, R, er, "rstd")
    check(y, Y, np.abs(G) * (R * em)[:, None] * (1 + rel) + rel * np.abs(Y - B) + 2 * E * np.abs(Y), "y")
    m64, r64 = f64(mean), f64(rstd)
    DX, DG, DB = dense.layer_norm_backward(D, X, G, m64, r64)
    dx, dg, db = moe.layer_norm_backward(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd)
    XH, GG = (X - m64[:, None]) * r64[:, None], D * G
    eg = 4 * np.abs(GG) + 52 * np.abs(GG).mean(1, keepdims=True) + \
        np.abs(XH) * 58 * np.abs(GG * XH).mean(1, keepdims=True)
    check(dx, DX, r64[:, None] * E * eg, "dx")
    check(dg, DG, (rows + 8) * E * np.abs(D * XH).sum(0), "dgamma")
    check(db, DB, (rows + 8) * E * np.abs(D).sum(0), "dbeta")
