"""Operands that end where an allocation ends: boxes of the products' copies reach behind the last rows, which must read
nothing there, whatever lies behind (elements out of bounds are zeros).  Segments of one row at an operand's end, with maps
that the device builds for each segment, are the sharpest case: none of the rows behind the first belongs to them."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_dense import acc_bound, check, dev_offsets, f64, offsets_of

pytestmark = pytest.mark.gpu

PAGE = 2 << 20


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()
    yield
    torch.cuda.empty_cache()


def at_the_end(t):
    """A copy of t in the last bytes of an allocation of whole pages of its own."""
    n = t.numel() * t.element_size()
    whole = max(-(-n // PAGE), 6) * PAGE                      # 10 MB and more: a block of its own
    buf = torch.zeros(whole, dtype=torch.uint8, device="cuda")
    out = buf[whole - n:].view(t.dtype).view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("counts,K,N", [([895 - 2, 2], 496, 920), ([17, 263, 20, 0, 2], 496, 920), ([1] * 40, 336, 1536),
                                        ([2000, 1], 72, 136), ([130, 133, 1], 496, 920), ([1], 8, 8), ([63, 1], 2048, 1024)])
@pytest.mark.parametrize("before", [0, 5])
def test_segments_at_the_end_of_an_allocation(counts, K, N, before):
    torch.cuda.empty_cache()
    gen = torch.Generator().manual_seed(K + before)
    off = offsets_of(counts, before)
    M, E = off[-1], len(counts)
    x, dy = torch.randn((M, K), generator=gen).bfloat16(), torch.randn((M, N), generator=gen).bfloat16()
    w = (torch.randn((E, N, K), generator=gen) * K ** -0.5).bfloat16()
    xd, dyd, wd, o = at_the_end(x), at_the_end(dy), at_the_end(w), dev_offsets(off)
    X, D, W = f64(x), f64(dy), f64(w)
    inside = slice(before, M)
    y = moe.grouped_mm(xd, wd, o)
    check(y[inside], dense.grouped_mm(X, W, off)[inside],
          acc_bound(K, dense.grouped_mm(np.abs(X), np.abs(W), off)[inside]), "y")
    DX, DW = dense.grouped_mm_backward(D, X, W, off)
    SDX, SDW = dense.grouped_mm_backward(np.abs(D), np.abs(X), np.abs(W), off)
    for dw_dtype in (torch.bfloat16, torch.float32):
        dx, dw = moe.grouped_mm_backward(dyd, xd, wd, o, dw_dtype=dw_dtype)
        check(dx[inside], DX[inside], acc_bound(N, SDX[inside]), "dx")
        check(dw, DW, acc_bound(max(counts), SDW), "dw")
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 2, 33, 131, 133, 300])
def test_dense_rows_at_the_end_of_an_allocation(M):
    torch.cuda.empty_cache()
    K, N = 496, 264
    gen = torch.Generator().manual_seed(M)
    x, dy = torch.randn((M, K), generator=gen).bfloat16(), torch.randn((M, N), generator=gen).bfloat16()
    w = (torch.randn((N, K), generator=gen) * K ** -0.5).bfloat16()
    xd, dyd, wd = at_the_end(x), at_the_end(dy), at_the_end(w)
    X, D, W = f64(x), f64(dy), f64(w)
    check(moe.linear(xd, wd), X @ W.T, acc_bound(K, np.abs(X) @ np.abs(W).T), "y")
    dx, dw, _ = moe.linear_backward(dyd, xd, wd)
    check(dx, D @ W, acc_bound(N, np.abs(D) @ np.abs(W)), "dx")
    check(dw, D.T @ X, acc_bound(M, np.abs(D).T @ np.abs(X)), "dw")
    torch.cuda.synchronize()
