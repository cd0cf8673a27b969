"""Short products whose rows end inside the epilogue's 32-row pieces, many times over: every call of the loop is
compared, the first against FP64 in every element, the others with the first bit by bit (an order of additions
is fixed).  With 64 values to add, an epilogue follows the next as fast as it can, and every warp stores whole and
partial pieces in turn from the same two buffers."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_dense import acc_bound, check, dev_offsets, f64, offsets_of, rand

pytestmark = pytest.mark.gpu

CALLS = 400


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def every_call_agrees(call, outs):
    """Runs ``call`` CALLS times, its outputs refilled in between, and counts the elements that differ from the
    first call's on the device."""
    call()
    first = [t.clone() for t in outs]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(CALLS):
        for t in outs:
            t.fill_(7.0)
        call()
        for t, f in zip(outs, first):
            wrong += (t != f).sum()
    assert int(wrong) == 0
    return first


# rows of a segment are 32 n + 8: from 40 (tiles of 64 rows on single CTAs) to 264 (pairs)
GROUPED = [([40] * 24, 64, 2048), ([72] * 24, 64, 2048), ([104, 8, 40, 0, 200] * 8, 64, 1032),
           ([136] * 16, 64, 4096), ([264] * 12, 64, 2568), ([1032, 40, 520], 64, 4096)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_segments_that_end_inside_a_piece(case, dtype):
    counts, K, N = GROUPED[case]
    gen = torch.Generator().manual_seed(700 + case)
    off = offsets_of(counts)
    M, E = off[-1], len(counts)
    x, w = rand(gen, M, K, dtype=dtype), rand(gen, E, N, K, dtype=dtype, scale=K ** -0.5)
    dy = rand(gen, M, K, dtype=dtype)
    v = rand(gen, E, K, N, dtype=dtype, scale=K ** -0.5)           # dx = dy v: 64 values to add, N columns
    xd, wd, dyd, vd, o = x.cuda(), w.cuda(), dy.cuda(), v.cuda(), dev_offsets(off)
    y = torch.empty((M, N), dtype=dtype, device="cuda")
    dx = torch.empty((M, N), dtype=dtype, device="cuda")
    ws = torch.empty(max(moe.grouped_mm_workspace_bytes(E), moe.grouped_mm_backward_workspace_bytes(M, N, E, K)),
                     dtype=torch.uint8, device="cuda")
    any_x = torch.empty((M, N), dtype=dtype, device="cuda")

    def call():
        moe.grouped_mm(xd, wd, o, out=y, ws=ws)
        moe.grouped_mm_backward(dyd, any_x, vd, o, need_dw=False, dx=dx, ws=ws)

    got_y, got_dx = every_call_agrees(call, (y, dx))
    assert moe.status_read(ws) == moe.OK
    X, W, D, V = f64(x), f64(w), f64(dy), f64(v)
    check(got_y, dense.grouped_mm(X, W, off), acc_bound(K, dense.grouped_mm(np.abs(X), np.abs(W), off)), "y")
    Vt = V.transpose(0, 2, 1)
    check(got_dx, dense.grouped_mm(D, Vt, off), acc_bound(K, dense.grouped_mm(np.abs(D), np.abs(Vt), off)), "dx")


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N", [(40, 20480), (72, 12296), (104, 8192), (328, 8192), (1032, 8192), (2088, 4104)])
def test_linear_rows_that_end_inside_a_piece(M, N, act):
    K = 64
    gen = torch.Generator().manual_seed(M + N)
    x, w, res = rand(gen, M, K), rand(gen, N, K, scale=K ** -0.5), rand(gen, M, N, scale=3.0)
    bias = torch.randn(N, generator=gen)
    xd, wd, rd, bd = x.cuda(), w.cuda(), res.cuda(), bias.cuda()
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dx = torch.empty_like(y)
    vd = rand(gen, K, N, scale=K ** -0.5).cuda()
    kept = []

    def call():
        kept[:] = [moe.linear(xd, wd, bias=bd, act=act, residual=rd, save_z=True, out=y)[1]]
        moe.linear_backward(xd, y, vd, need_dw=False, dx=dx)

    call()
    z0 = kept[0].clone()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")

    def call_and_compare_z():
        call()
        wrong.add_((kept[0] != z0).sum())

    got_y, got_dx = every_call_agrees(call_and_compare_z, (y, dx))
    assert int(wrong) == 0
    X, W = f64(x), f64(w)
    Y, Z = dense.linear(X, W, f64(bias), act, f64(res))
    ez = acc_bound(K + 1, np.abs(X) @ np.abs(W).T + np.abs(f64(bias)))
    ey = ez if act == "none" else 1.13 * ez + 2.0 ** -20 * np.abs(Z)
    check(z0, Z, ez, "z")
    check(got_y, Y, ey + 2.0 ** -24 * (np.abs(Y) + ey), "y")
    V = f64(vd)
    check(got_dx, X @ V, acc_bound(K, np.abs(X) @ np.abs(V)), "dx")
