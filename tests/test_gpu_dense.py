"""The 16-bit products on the GPU against the FP64 oracle: products grouped by expert, the dense
product with its epilogue, and their gradients.

Bounds.  Operands are exact in FP32 and so is every product of two of them (at most 22 bits).  The
tensor cores add R products in FP32; each addition may lose up to one unit in the last place
(2^-23) of a partial sum no larger than S = sum |a b|, so a sum is off by at most (R + 2) 2^-23 S.
Rounding to the output type adds half a step: u |value| (bf16 2^-8, fp16 2^-11, fp32 2^-24), or half
the smallest subnormal step.  The activations' FP32 evaluation is off by at most 2^-20 |z| and their
slopes by at most 2^-19 (a few roundings, exp within 2 + 1.16 |x| units, and |x| e^-|x| < 0.37); their
slope is below 1.13.  dz is rounded to the operands' type before the backward products."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def acc_bound(R, S):
    return (R + 2) * 2.0 ** -23 * S


def check(got, want, err, what):
    """|got - want| <= err + the output's rounding, elementwise."""
    g = f64(got)
    assert np.isfinite(g).all(), what
    bound = err + U[got.dtype] * (np.abs(want) + err) + TINY[got.dtype]
    worst = np.max((np.abs(g - want) - bound) if g.size else np.array([-1.0]))
    assert worst <= 0, (what, worst, np.unravel_index(np.argmax(np.abs(g - want) - bound), g.shape))


def offsets_of(counts, first=0):
    return [first] + [first + int(v) for v in np.cumsum(counts)]


def dev_offsets(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


GROUPED = [
    # counts, K, N, rows before the first segment, rows behind the last
    ([1], 8, 8, 0, 0),
    ([1], 64, 256, 0, 0),
    ([5, 0, 3], 64, 64, 0, 0),
    ([0, 0, 7], 72, 136, 3, 5),
    ([300, 1, 0, 129, 256], 200, 264, 1, 9),
    ([64, 63, 65, 128], 512, 520, 0, 0),
    ([700], 1032, 24, 0, 1),
    ([17] * 40, 24, 1000, 0, 0),
    ([2, 0] * 100, 128, 256, 0, 0),
    ([1025, 511], 320, 776, 7, 0),
    # many rows, few tiles: dw's rows in parts
    ([4000, 0], 264, 264, 2, 3),
    ([3700, 0, 5, 1300, 64], 72, 40, 0, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_forward_and_gradients(case, dtype):
    counts, K, N, before, behind = GROUPED[case]
    gen = torch.Generator().manual_seed(100 + case)
    off = offsets_of(counts, before)
    M, E = off[-1] + behind, len(counts)
    x, dy = rand(gen, M, K, dtype=dtype), rand(gen, M, N, dtype=dtype)
    w = rand(gen, E, N, K, dtype=dtype, scale=K ** -0.5)
    # rows outside the segments: never used, whatever they hold
    for t in (x, dy):
        t[:before] = float("nan")
        t[off[-1]:] = float("inf")
    X, W, D = f64(x), f64(w), f64(dy)
    xd, wd, dyd, o = x.cuda(), w.cuda(), dy.cuda(), dev_offsets(off)
    inside = slice(before, off[-1])
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(moe.grouped_mm_backward_workspace_bytes(M, K, E, N), dtype=torch.uint8, device="cuda")
    y = moe.grouped_mm(xd, wd, o, out=out, ws=ws)
    assert moe.status_read(ws) == moe.OK
    assert y.data_ptr() == out.data_ptr()
    check(y[inside], dense.grouped_mm(X, W, off)[inside],
          acc_bound(K, dense.grouped_mm(np.abs(X), np.abs(W), off)[inside]), "y")
    assert (y[:before] == 7).all() and (y[off[-1]:] == 7).all()
    dx = torch.full((M, K), 7.0, dtype=dtype, device="cuda")
    DX, DW = dense.grouped_mm_backward(D, X, W, off)
    SDX, SDW = dense.grouped_mm_backward(np.abs(D), np.abs(X), np.abs(W), off)
    rows = max(counts)
    got_dx, dw = moe.grouped_mm_backward(dyd, xd, wd, o, dx=dx, ws=ws)
    assert moe.status_read(ws) == moe.OK
    check(got_dx[inside], DX[inside], acc_bound(N, SDX[inside]), "dx")
    assert (got_dx[:before] == 7).all() and (got_dx[off[-1]:] == 7).all()
    check(dw, DW, acc_bound(rows, SDW), "dw")
    none, dw32 = moe.grouped_mm_backward(dyd, xd, wd, o, need_dx=False, dw_dtype=torch.float32)
    assert none is None and dw32.dtype == torch.float32
    check(dw32, DW, acc_bound(rows, SDW), "dw fp32")
    dx2, none = moe.grouped_mm_backward(dyd, xd, wd, o, need_dw=False)
    assert none is None and torch.equal(dx2[inside], got_dx[inside])


def test_nan_and_inf_stay_in_their_segment():
    """A row of NaN or Inf spoils its own output row and its expert's dw, nothing else."""
    gen = torch.Generator().manual_seed(5)
    counts, K, N = [70, 33, 90], 136, 264
    off = offsets_of(counts)
    x, dy, w = rand(gen, off[-1], K), rand(gen, off[-1], N), rand(gen, 3, N, K)
    bad = off[1] + 4
    x[bad], dy[bad] = float("nan"), float("inf")
    clean_x, clean_dy = x.clone(), dy.clone()
    clean_x[bad], clean_dy[bad] = 0, 0
    o = dev_offsets(off)
    args = (x.cuda(), w.cuda(), o)
    y, y0 = moe.grouped_mm(*args), moe.grouped_mm(clean_x.cuda(), w.cuda(), o)
    dx, dw = moe.grouped_mm_backward(dy.cuda(), *args)
    dx0, dw0 = moe.grouped_mm_backward(clean_dy.cuda(), clean_x.cuda(), w.cuda(), o)
    keep = torch.ones(off[-1], dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[bad]).all()
    assert torch.equal(dx[keep], dx0[keep])
    assert torch.equal(dw[0], dw0[0]) and torch.equal(dw[2], dw0[2]) and torch.isnan(dw[1]).all()
    # an expert's weights of NaN spoil its own rows
    w[1] = float("nan")
    y = moe.grouped_mm(clean_x.cuda(), w.cuda(), o)
    other = torch.ones(off[-1], dtype=torch.bool)
    other[off[1]:off[2]] = False
    assert torch.equal(y[other], y0[other]) and torch.isnan(y[~other]).all()
    dx = moe.grouped_mm_backward(clean_dy.cuda(), clean_x.cuda(), w.cuda(), o, need_dw=False)[0]
    assert torch.equal(dx[other], dx0[other])


def test_no_rows():
    w = torch.randn(3, 16, 24, device="cuda").bfloat16()
    x = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert moe.grouped_mm(x, w, o).shape == (0, 16)
    dx, dw = moe.grouped_mm_backward(dy, x, w, o)
    assert dx.shape == (0, 24) and (dw == 0).all()
    # rows, but every expert empty
    x1, dy1 = torch.ones((5, 24), device="cuda").bfloat16(), torch.ones((5, 16), device="cuda").bfloat16()
    out = torch.full((5, 16), 3.0, device="cuda").bfloat16()
    assert (moe.grouped_mm(x1, w, o + 2, out=out) == 3).all()
    assert (moe.grouped_mm_backward(dy1, x1, w, o + 2, need_dx=False)[1] == 0).all()
    assert moe.linear(x, w[0]).shape == (0, 16)
    dx, dw, db = moe.linear_backward(dy, x, w[0], z=dy, act="silu", bias=True)
    assert dx.shape == (0, 24) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("off", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 2, 4, 9], [5, 4, 6, 8]])
def test_bad_offsets_are_reported_and_touch_nothing(off):
    x, w = torch.ones((8, 64), device="cuda").bfloat16(), torch.ones((3, 64, 64), device="cuda").bfloat16()
    out = torch.full((8, 64), 3.0, device="cuda").bfloat16()
    ws = torch.empty(moe.grouped_mm_backward_workspace_bytes(8, 64, 3, 64), dtype=torch.uint8, device="cuda")
    y = moe.grouped_mm(x, w, dev_offsets(off), out=out, ws=ws)
    assert moe.status_read(ws) == moe.ERR_ARG and moe.last_device_status() == moe.ERR_ARG
    assert (y == 3).all()
    dx, dw = moe.grouped_mm_backward(x, x, w, dev_offsets(off), dx=out, ws=ws)
    assert moe.status_read(ws) == moe.ERR_ARG and (dx == 3).all() and (dw == 0).all()
    # the same workspace serves the next call
    moe.grouped_mm(x, w, dev_offsets([0, 2, 4, 8]), out=out, ws=ws)
    assert moe.status_read(ws) == moe.OK and (out == 64).all()


LINEAR = [
    # M, K, N, act, bias, residual, z
    (1, 8, 8, "none", False, False, False),
    (1, 5120, 512, "none", True, True, False),
    (2, 72, 1000, "silu", True, False, True),
    (3, 136, 264, "gelu", False, True, True),
    (7, 2568, 136, "relu", True, True, False),
    (16, 640, 2560, "gelu_tanh", True, True, True),
    (31, 1032, 320, "silu", False, False, False),
    (33, 256, 72, "gelu", True, False, False),
    (65, 520, 776, "none", True, False, True),
    (129, 192, 1288, "gelu_tanh", False, True, True),
    (256, 256, 256, "relu", True, True, True),
    (300, 1000, 136, "silu", True, True, True),
    (1030, 72, 520, "gelu", True, True, True),
    # long reductions, few tiles: in parts forward, in dx, in dw
    (290, 16008, 520, "gelu", True, True, True),
    (600, 16008, 264, "gelu", True, True, True),
    (257, 16000, 264, "none", False, False, False),
    (520, 40, 16008, "silu", False, False, False),
    (2500, 264, 264, "relu", True, False, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(LINEAR)))
def test_linear_forward_and_gradients(case, dtype):
    M, K, N, act, has_bias, has_res, save_z = LINEAR[case]
    gen = torch.Generator().manual_seed(200 + case)
    x, w = rand(gen, M, K, dtype=dtype), rand(gen, N, K, dtype=dtype, scale=2.0 * K ** -0.5)
    bias = torch.randn(N, generator=gen) if has_bias else None
    res = rand(gen, M, N, dtype=dtype, scale=3.0) if has_res else None
    dy = rand(gen, M, N, dtype=dtype)
    X, W, D = f64(x), f64(w), f64(dy)
    Y, Z = dense.linear(X, W, f64(bias) if has_bias else None, act, f64(res) if has_res else None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ws = torch.empty(moe.linear_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    got = moe.linear(cu(x), cu(w), bias=cu(bias), act=act, residual=cu(res), save_z=save_z, ws=ws)
    assert moe.status_read(ws) == moe.OK
    y, z = got if save_z else (got, None)
    ez = acc_bound(K + 1, np.abs(X) @ np.abs(W).T + (np.abs(f64(bias)) if has_bias else 0.0))
    ey = ez if act == "none" else 1.13 * ez + 2.0 ** -20 * np.abs(Z)
    if has_res:
        ey = ey + 2.0 ** -24 * (np.abs(Y) + ey)
    check(y, Y, ey, "y")
    if save_z:
        check(z, Z, ez, "z")
    if has_res:          # the residual updated in place
        r2 = res.cuda()
        moe.linear(cu(x), cu(w), bias=cu(bias), act=act, residual=r2, out=r2)
        assert torch.equal(r2, y)
    # backward at the rounded z
    zr = torch.from_numpy(Z).to(dtype)
    DX, DW, DB = dense.linear_backward(D, X, W, f64(zr), act)
    wsb = torch.empty(moe.linear_backward_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    dx, dw, db = moe.linear_backward(cu(dy), cu(x), cu(w), z=None if act == "none" else cu(zr), act=act, bias=True,
                                     ws=wsb)
    assert moe.status_read(wsb) == moe.OK
    if act == "none":
        DZ, edz, edz32 = D, np.zeros_like(D), np.zeros_like(D)
    else:
        DZ = D * dense.act_slope(f64(zr), act)
        edz32 = 2.0 ** -19 * np.abs(D) + 2.0 ** -24 * np.abs(DZ)
        edz = edz32 + U[dtype] * (np.abs(DZ) + edz32) + TINY[dtype]
    A = np.abs(DZ) + edz
    check(dx, DX, edz @ np.abs(W) + acc_bound(N, A @ np.abs(W)), "dx")
    check(dw, DW, edz.T @ np.abs(X) + acc_bound(M, A.T @ np.abs(X)), "dw")
    check(db, DB, edz32.sum(0) + M * 2.0 ** -24 * A.sum(0), "db")
    _, dw32, _ = moe.linear_backward(cu(dy), cu(x), cu(w), z=None if act == "none" else cu(zr), act=act,
                                     need_dx=False, dw_dtype=torch.float32)
    check(dw32, DW, edz.T @ np.abs(X) + acc_bound(M, A.T @ np.abs(X)), "dw fp32")


@pytest.mark.parametrize("act", dense.ACTIVATIONS)
def test_activation_extremes(act):
    """Far arguments: no NaN out of finite z, the limits reached, NaN kept."""
    z = torch.tensor([-6e4, -300.0, -90.0, -20.0, -1e-7, 0.0, 1e-7, 20.0, 90.0, 300.0, 6e4])
    n = 16
    zz = torch.zeros((1, n))
    zz[0, :11] = z
    x = torch.zeros((1, 8), dtype=torch.float16, device="cuda")
    w = torch.zeros((n, 8), dtype=torch.float16, device="cuda")
    bias = zz[0].cuda()
    y = f64(moe.linear(x, w, bias=bias, act=act))
    assert np.isfinite(y).all()
    want = dense.act(f64(zz.half()), act)
    with np.errstate(over="ignore"):
        np.testing.assert_allclose(y, want, rtol=2.0 ** -10, atol=2.0 ** -24)
    dy = torch.ones((1, n), dtype=torch.float16, device="cuda")
    db = f64(moe.linear_backward(dy, x, w, z=zz.half().cuda(), act=act, bias=True)[2])
    with np.errstate(over="ignore"):
        np.testing.assert_allclose(db, dense.act_slope(f64(zz.half()), act)[0], rtol=0, atol=2.0 ** -19)
    big = torch.tensor([[-3e38, 3e38] + [0.0] * 6]).bfloat16().cuda()     # squares and cubes overflow
    one, w8 = torch.ones((1, 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((8, 8), device="cuda").bfloat16()
    db = f64(moe.linear_backward(one, one, w8, z=big, act=act, bias=True)[2])
    np.testing.assert_allclose(db[:2], [1, 1] if act == "none" else [0, 1], atol=2.0 ** -19)
    bias[3] = float("nan")
    assert torch.isnan(moe.linear(x, w, bias=bias, act=act)[0, 3])


def test_gradients_against_differences():
    """dx of linear and of grouped_mm against central differences of the kernels' own forward: for a
    linear map the difference is exact up to the roundings of the two outputs."""
    gen = torch.Generator().manual_seed(9)
    M, K, N = 20, 64, 48
    x, w, dy = rand(gen, M, K, dtype=torch.float16), rand(gen, 2, N, K, dtype=torch.float16, scale=0.125), \
        rand(gen, M, N, dtype=torch.float16)
    o = dev_offsets([0, 9, M])
    v = rand(gen, M, K, dtype=torch.float16)
    dx, dw = moe.grouped_mm_backward(dy.cuda(), x.cuda(), w.cuda(), o)
    dxl, dwl, _ = moe.linear_backward(dy.cuda(), x.cuda(), w[0].cuda())
    # x +- 2^-4 v is exact here only up to its own rounding: the step taken is the rounded one
    xp, xm = (x + 0.0625 * v), (x - 0.0625 * v)
    step = f64(xp) - f64(xm)
    for plus, minus, g, W in ((moe.grouped_mm(xp.cuda(), w.cuda(), o), moe.grouped_mm(xm.cuda(), w.cuda(), o), dx, None),
                              (moe.linear(xp.cuda(), w[0].cuda()), moe.linear(xm.cuda(), w[0].cuda()), dxl, w[0])):
        p, m = f64(plus), f64(minus)
        lhs = ((p - m) * f64(dy)).sum()
        rhs = (step * f64(g)).sum()
        # the outputs' half steps and the gradient's half step
        tol = (2.0 ** -11 * (np.abs(p) + np.abs(m)) * np.abs(f64(dy))).sum() + \
            (2.0 ** -11 * np.abs(f64(g)) * np.abs(step)).sum() + 1e-3
        assert abs(lhs - rhs) <= tol, (lhs, rhs, tol)


def test_outputs_and_workspaces_live_on_the_stream_given():
    """What a call on another stream allocates is not handed out again while that stream still needs it,
    even though the caller drops it at once and the current stream goes on allocating."""
    x = torch.randn((4096, 2048), device="cuda").bfloat16()
    w = torch.randn((2048, 2048), device="cuda").bfloat16()
    g = torch.ones(2048, device="cuda")
    side = torch.cuda.Stream()
    want = moe.linear(x, w, act="silu", save_z=True)
    grads = moe.linear_backward(x, x, w, z=want[1], act="silu", bias=True)
    y, m, r = moe.layer_norm(x, g, g, stats=True)
    ng = moe.layer_norm_backward(x, x, g, m, r)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    kept = []
    for _ in range(6):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)               # the side stream is behind the host
        for i in range(3):
            got = (moe.linear_backward(x, x, w, z=want[1], act="silu", bias=True, stream=side),
                   moe.layer_norm_backward(x, x, g, m, r, stream=side))
            if i == 2:
                kept.append(got)
            del got
        junk = [torch.full((4096, 2048), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(6)]
        del junk
    torch.cuda.synchronize()
    for lin, nrm in kept:
        assert all(torch.equal(a, b) for a, b in zip(lin, grads))
        assert all(torch.equal(a, b) for a, b in zip(nrm, ng))


def test_many_experts():
    """The largest number of experts, most of them without rows."""
    gen = torch.Generator().manual_seed(21)
    E, K, N = 1024, 72, 40
    counts = [0] * E
    for e, c in ((0, 1), (1, 3), (31, 70), (32, 2), (500, 300), (1023, 65)):
        counts[e] = c
    off = offsets_of(counts)
    x, dy = rand(gen, off[-1], K), rand(gen, off[-1], N)
    w = rand(gen, E, N, K, scale=K ** -0.5)
    ws = torch.full((moe.grouped_mm_backward_workspace_bytes(off[-1], K, E, N),), 255, dtype=torch.uint8, device="cuda")
    args = (x.cuda(), w.cuda(), dev_offsets(off))
    y = moe.grouped_mm(*args, ws=ws)
    assert moe.status_read(ws) == moe.OK
    dx, dw = moe.grouped_mm_backward(dy.cuda(), *args, ws=ws)
    assert moe.status_read(ws) == moe.OK
    X, W, D = f64(x), f64(w), f64(dy)
    check(y, dense.grouped_mm(X, W, off), acc_bound(K, dense.grouped_mm(np.abs(X), np.abs(W), off)), "y")
    DX, DW = dense.grouped_mm_backward(D, X, W, off)
    SDX, SDW = dense.grouped_mm_backward(np.abs(D), np.abs(X), np.abs(W), off)
    check(dx, DX, acc_bound(N, SDX), "dx")
    check(dw, DW, acc_bound(300, SDW), "dw")


def test_workspace_contents_do_not_matter():
    """The same results from workspaces full of ones and of zeros."""
    gen = torch.Generator().manual_seed(22)
    off = offsets_of([40, 0, 90, 3])
    x, w = rand(gen, off[-1], 128).cuda(), rand(gen, 4, 264, 128).cuda()
    dy, o = rand(gen, off[-1], 264).cuda(), dev_offsets(off)
    got = []
    for fill in (0, 255):
        ws = lambda n: torch.full((n,), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        a, b = ws(moe.grouped_mm_backward_workspace_bytes(133, 128, 4, 264)), ws(moe.linear_backward_workspace_bytes(133, 128, 264))
        got.append((moe.grouped_mm(x, w, o, ws=a), *moe.grouped_mm_backward(dy, x, w, o, ws=a),
                    moe.linear(x, w[0], ws=ws(moe.linear_workspace_bytes(133, 128, 264))),
                    *moe.linear_backward(dy, x, w[0], z=dy, act="relu", bias=True, ws=b)))
        assert moe.status_read(a) == moe.OK and moe.status_read(b) == moe.OK
    assert all(torch.equal(p, q) for p, q in zip(*got))


def test_parts_are_joined_in_order():
    """Products whose reduction is shared by several pairs: one launch more, the same bits every time and
    from a captured graph, whatever the workspace held; bad offsets leave zeros in dw."""
    gen = torch.Generator().manual_seed(23)
    x, w, res = rand(gen, 600, 16008).cuda(), rand(gen, 264, 16008, scale=0.01).cuda(), rand(gen, 600, 264).cuda()
    a, b, v = rand(gen, 4000, 264).cuda(), rand(gen, 4000, 136).cuda(), rand(gen, 2, 136, 264).cuda()
    o = dev_offsets([0, 3000, 4000])
    n1, n2 = moe.linear_workspace_bytes(600, 16008, 264), moe.linear_backward_workspace_bytes(4000, 264, 136)
    n3 = moe.grouped_mm_backward_workspace_bytes(4000, 264, 2, 136)

    def run(fill):
        ws = [torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in (n1, n2, n3)]
        y = moe.linear(x, w, residual=res, act="silu", ws=ws[0])
        launches = [moe.last_launch_count()]
        dx, dw, _ = moe.linear_backward(b, a, v[0], ws=ws[1])
        launches.append(moe.last_launch_count())
        dx2, dw2 = moe.grouped_mm_backward(b, a, v, o, ws=ws[2], dw_dtype=torch.float32)
        launches.append(moe.last_launch_count())
        return [y, dx, dw, dx2, dw2], launches, ws

    first, launches, _ = run(0)
    assert launches == [2, 4, 4]
    second = run(255)[0]
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third, _, ws = run(255)
    for t in third:
        t.fill_(float("nan"))
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(first, third))
    ws = torch.full((n3,), 255, dtype=torch.uint8, device="cuda")
    dw = moe.grouped_mm_backward(b, a, v, dev_offsets([0, 4000, 3000]), ws=ws, need_dx=False)[1]
    assert moe.status_read(ws) == moe.ERR_ARG and (dw == 0).all()


def test_another_stream_and_graph_replay():
    gen = torch.Generator().manual_seed(11)
    off = offsets_of([40, 0, 90, 3])
    x, w = rand(gen, off[-1], 128).cuda(), rand(gen, 4, 264, 128).cuda()
    dy, o = rand(gen, off[-1], 264).cuda(), dev_offsets(off)
    bias = torch.randn(264, device="cuda")
    y0 = moe.grouped_mm(x, w, o)
    g0 = moe.grouped_mm_backward(dy, x, w, o)
    l0 = moe.linear(x, w[0], bias=bias, act="gelu", residual=dy)
    b0 = moe.linear_backward(dy, x, w[0], z=dy, act="gelu", bias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = moe.grouped_mm(x, w, o, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = moe.grouped_mm(x, w, o)
        g2 = moe.grouped_mm_backward(dy, x, w, o)
        l2 = moe.linear(x, w[0], bias=bias, act="gelu", residual=dy)
        b2 = moe.linear_backward(dy, x, w[0], z=dy, act="gelu", bias=True)
    for _ in range(3):
        for t in (y2, *g2, l2, *b2):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y0, *g0, l0, *b0), (y2, *g2, l2, *b2)):
            assert torch.equal(a, b)
    # a replay follows the offsets' new contents
    new = offsets_of([3, 90, 0, 40])
    o.copy_(dev_offsets(new))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, moe.grouped_mm(x, w, o))


def test_repeated_calls_agree():
    """Every output has one fixed order of additions."""
    gen = torch.Generator().manual_seed(12)
    off = offsets_of([100, 37, 260, 1])
    x, w, dy = rand(gen, off[-1], 776).cuda(), rand(gen, 4, 520, 776).cuda(), rand(gen, off[-1], 520).cuda()
    o = dev_offsets(off)
    first = None
    for _ in range(5):
        got = (moe.grouped_mm(x, w, o), *moe.grouped_mm_backward(dy, x, w, o), moe.linear(x[:9], w[0]),
               *moe.linear_backward(dy, x, w[0], z=dy, act="silu", bias=True))
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
