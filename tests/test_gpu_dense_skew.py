"""Grouped products whose rows are far from evenly spread: the shape of the kernels and the parts of dw are chosen for the
mean segment, on the host, and have to hold for any spread of the rows."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_dense import acc_bound, check, dev_offsets, f64, offsets_of, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


SPREADS = [
    # counts, K, N
    ([1] * 60 + [901], 136, 264),                # a mean of 16 rows: tiles of 16, 57 of them in one segment
    ([0] * 50 + [1501] + [2] * 12, 264, 136),    # nearly all rows with one expert of 63
    ([2048] + [0] * 63, 72, 520),                # all of them
    ([0, 0, 5000, 3], 264, 264),                 # dw's parts: long steps for one expert, none for the others
    ([1] * 200 + [400] * 2 + [0] * 54, 64, 1032),
]


@pytest.mark.parametrize("case", range(len(SPREADS)))
def test_skewed_segments(case):
    counts, K, N = SPREADS[case]
    gen = torch.Generator().manual_seed(800 + case)
    off = offsets_of(counts)
    M, E = off[-1], len(counts)
    x, dy, w = rand(gen, M, K), rand(gen, M, N), rand(gen, E, N, K, scale=K ** -0.5)
    X, D, W = f64(x), f64(dy), f64(w)
    xd, dyd, wd, o = x.cuda(), dy.cuda(), w.cuda(), dev_offsets(off)
    ws = torch.full((moe.grouped_mm_backward_workspace_bytes(M, K, E, N),), 255, dtype=torch.uint8, device="cuda")
    y = moe.grouped_mm(xd, wd, o, ws=ws)
    assert moe.status_read(ws) == moe.OK
    check(y, dense.grouped_mm(X, W, off), acc_bound(K, dense.grouped_mm(np.abs(X), np.abs(W), off)), "y")
    dx, dw = moe.grouped_mm_backward(dyd, xd, wd, o, ws=ws, dw_dtype=torch.float32)
    assert moe.status_read(ws) == moe.OK
    DX, DW = dense.grouped_mm_backward(D, X, W, off)
    SDX, SDW = dense.grouped_mm_backward(np.abs(D), np.abs(X), np.abs(W), off)
    check(dx, DX, acc_bound(N, SDX), "dx")
    check(dw, DW, acc_bound(max(counts), SDW), "dw")
