"""Layer norm forward and backward on the GPU against the FP64 oracle.

Bounds, e = 2^-24 (FP32 half step).  A thread adds at most 32 values, then 5 + 5 shuffle steps follow:
a row sum passes through fewer than 48 roundings, so mean is off by at most 48 e mean|x| (+ e |mean|) and
the mean of squares by 50 e of itself plus the square of the mean's error; rstd's relative error is half of
that plus 4 e.  y inherits |gamma| rstd times the mean's error and 40 e of |y - beta|, then one rounding of the
output type.  Backward takes the statistics as inputs: xh is off by 2 e |xh|, g by e |g|, the row means
by 50 e mean|g| and 54 e mean|g xh|.  A column sum of `rows` terms passes through at most rows + 2 additions."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: E}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, err, what):
    g = f64(got)
    assert np.isfinite(g).all(), what
    bound = err + U[got.dtype] * (np.abs(want) + err) + TINY[got.dtype]
    d = np.abs(g - want) - bound
    assert d.max() <= 0, (what, d.max(), np.unravel_index(np.argmax(d), d.shape))


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (9, 63), (130, 64), (33, 250), (4, 256), (7, 1000), (65, 1016), (3, 1017),
          (5, 2048), (4, 2049), (9, 2571), (700, 3001), (16, 5120), (3, 8192), (2, 8200), (3, 8193), (2, 16384), (3, 16386), (2, 28671),
          (2, 28672), (700, 40), (1201, 96)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(shape, rms, dtype):
    rows, cols = shape
    gen = torch.Generator().manual_seed(rows * 31 + cols)
    x = (torch.randn((rows, cols), generator=gen) * 3 + 0.7).to(dtype)
    dy = torch.randn((rows, cols), generator=gen).to(dtype)
    gamma = 1 + 0.2 * torch.randn(cols, generator=gen)
    beta = None if rms else torch.randn(cols, generator=gen)
    X, D, G = f64(x), f64(dy), f64(gamma)
    B = 0.0 if rms else f64(beta)
    eps = 1e-2                     # a single column has variance 0
    epsr = float(np.float32(eps))
    Y, MEAN, R = dense.layer_norm(X, G, B if not rms else None, epsr, rms)
    y, mean, rstd = moe.layer_norm(x.cuda(), gamma.cuda(), None if rms else beta.cuda(), eps=eps, rms=rms, stats=True)
    em = np.zeros(rows) if rms else 48 * E * np.abs(X).mean(1) + E * np.abs(MEAN)
    er = R * (29 * E + 0.5 * (em * R) ** 2)
    if rms:
        assert mean is None
    else:
        check(mean, MEAN, em, "mean")
    check(rstd, R, er, "rstd")
    rel = (er / R)[:, None] + 8 * E
    check(y, Y, np.abs(G) * (R * em)[:, None] * (1 + rel) + rel * np.abs(Y - B) + 2 * E * np.abs(Y), "y")
    # backward, at the statistics the forward pass returned
    m64, r64 = (np.zeros(rows) if rms else f64(mean)), f64(rstd)
    DX, DG, DB = dense.layer_norm_backward(D, X, G, m64, r64, rms)
    dx, dg, db = moe.layer_norm_backward(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd, rms=rms)
    XH, GG = (X - m64[:, None]) * r64[:, None], D * G
    eg = 4 * np.abs(GG) + (0 if rms else 52 * np.abs(GG).mean(1, keepdims=True)) + \
        np.abs(XH) * 58 * np.abs(GG * XH).mean(1, keepdims=True)
    check(dx, DX, r64[:, None] * E * eg, "dx")
    check(dg, DG, (rows + 8) * E * np.abs(D * XH).sum(0), "dgamma")
    if rms:
        assert db is None
    else:
        check(db, DB, (rows + 8) * E * np.abs(D).sum(0), "dbeta")


@pytest.mark.parametrize("rms", [False, True])
def test_without_parameters_in_place_and_empty(rms):
    x = (torch.randn(37, 640) * 2 + 1).bfloat16().cuda()
    dy = torch.randn(37, 640).bfloat16().cuda()
    y, mean, rstd = moe.layer_norm(x, rms=rms, stats=True)
    ones, zeros = torch.ones(640, device="cuda"), torch.zeros(640, device="cuda")
    assert torch.equal(y, moe.layer_norm(x, ones, None if rms else zeros, rms=rms))
    x2 = x.clone()
    assert moe.layer_norm(x2, rms=rms, out=x2).data_ptr() == x2.data_ptr() and torch.equal(x2, y)
    dx, dg, db = moe.layer_norm_backward(dy, x, None, mean, rstd, rms=rms)
    assert dg is None and db is None
    dx1, dg1, db1 = moe.layer_norm_backward(dy, x, ones, mean, rstd, rms=rms)
    assert torch.equal(dx, dx1)
    dx2, dg2, db2 = moe.layer_norm_backward(dy, x, None, mean, rstd, rms=rms, need_params=True)
    assert torch.equal(dg2, dg1) and (rms or torch.equal(db2, db1))
    d = dy.clone()
    assert torch.equal(moe.layer_norm_backward(d, x, ones, mean, rstd, rms=rms, dx=d)[0], dx) and torch.equal(d, dx)
    e = torch.empty((0, 640), dtype=torch.bfloat16, device="cuda")
    y0, m0, r0 = moe.layer_norm(e, ones, rms=rms, stats=True)
    assert y0.shape == (0, 640) and r0.shape == (0,)
    dx0, dg0, db0 = moe.layer_norm_backward(e, e, ones, m0, r0, rms=rms)
    assert dx0.shape == (0, 640) and (dg0 == 0).all() and (rms or (db0 == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [3, 255, 1019, 5111, 9001, 20001])
@pytest.mark.parametrize("rows", [7, 700])
def test_in_place_rows_that_share_vectors(rows, cols, dtype):
    """Rows of odd length share 16-byte vectors with their neighbours; in place, a neighbour may already
    hold its result when a row is read."""
    x, dy = torch.randn(rows, cols).to(dtype).cuda(), torch.randn(rows, cols).to(dtype).cuda()
    g = torch.randn(cols).cuda()
    y, m, r = moe.layer_norm(x, g, stats=True)
    dx, dg, db = moe.layer_norm_backward(dy, x, g, m, r)
    for _ in range(3):
        x2, dy2 = x.clone(), dy.clone()
        assert torch.equal(moe.layer_norm(x2, g, out=x2), y)
        dx2, dg2, db2 = moe.layer_norm_backward(dy2, x, g, m, r, dx=dy2)
        assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


@pytest.mark.parametrize("cols", [640, 5111, 9000, 20001])
@pytest.mark.parametrize("rows", [5, 400])
def test_parameters_of_any_alignment(rows, cols):
    """gamma and beta need 4-byte alignment only."""
    x, dy = torch.randn(rows, cols).bfloat16().cuda(), torch.randn(rows, cols).bfloat16().cuda()
    buf = torch.randn(2, cols + 3).cuda()
    ref = None
    for shift in (0, 1, 3):
        g, b = torch.zeros(cols + shift).cuda()[shift:], torch.zeros(cols + shift).cuda()[shift:]
        g.copy_(buf[0, :cols])
        b.copy_(buf[1, :cols])
        assert g.data_ptr() % 16 == 4 * shift
        y, m, r = moe.layer_norm(x, g, b, stats=True)
        got = (y, m, r, *moe.layer_norm_backward(dy, x, g, m, r))
        ref = ref or got
        assert all(torch.equal(p, q) for p, q in zip(ref, got))


def test_large_offset_keeps_its_digits():
    """FP32 rows of 1000 + small noise: the variance is that of the noise (centred sums)."""
    gen = torch.Generator().manual_seed(3)
    x = 1000 + 0.01 * torch.randn((6, 3001), generator=gen)
    X = f64(x)
    Y, MEAN, R = dense.layer_norm(X, eps=0.0)
    y, mean, rstd = moe.layer_norm(x.cuda(), eps=0.0, stats=True)
    em = 48 * E * np.abs(X).mean(1) + E * np.abs(MEAN)
    er = R * (29 * E + 0.5 * (em * R) ** 2)
    check(rstd, R, er, "rstd")
    check(y, Y, (R * em)[:, None] * 1.01 + ((er / R)[:, None] + 8 * E) * np.abs(Y), "y")


def test_nan_stays_in_its_row():
    x = torch.randn(10, 777).cuda()
    x[4, 3] = float("nan")
    x[6, 5] = float("inf")
    y = moe.layer_norm(x)
    bad = torch.zeros(10, dtype=torch.bool)
    bad[[4, 6]] = True
    assert torch.isnan(y[bad]).any(1).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("cols", [640, 1001, 9000])
def test_graph_replay_and_other_stream(cols):
    x, dy = torch.randn(300, cols).bfloat16().cuda(), torch.randn(300, cols).bfloat16().cuda()
    g, b = torch.randn(cols).cuda(), torch.randn(cols).cuda()
    y, mean, rstd = moe.layer_norm(x, g, b, stats=True)
    ref = (y, mean, rstd, *moe.layer_norm_backward(dy, x, g, mean, rstd))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = moe.layer_norm(x, g, b, stats=True)
        got = (y2, m2, r2, *moe.layer_norm_backward(dy, x, g, m2, r2))
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ref, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3 = moe.layer_norm(x, g, b, stream=side)
    side.synchronize()
    assert torch.equal(y, y3)


def test_gradient_against_differences():
    """Directional derivatives of the FP32 kernels' own forward."""
    gen = torch.Generator().manual_seed(4)
    x, v, dy = (torch.randn((5, 96), generator=gen) for _ in range(3))
    g, b = torch.randn(96, generator=gen), torch.randn(96, generator=gen)
    y, mean, rstd = moe.layer_norm(x.cuda(), g.cuda(), b.cuda(), stats=True)
    dx, dg, db = moe.layer_norm_backward(dy.cuda(), x.cuda(), g.cuda(), mean, rstd)
    h = 2.0 ** -7
    f = lambda xx, gg, bb: (f64(moe.layer_norm(xx.cuda(), gg.cuda(), bb.cuda())) * f64(dy)).sum()  # noqa: E731
    # central difference: O(h^2) third derivatives (below 10 |v|^3 per row here) and 2^-22 of the outputs over h
    tol = 10 * h * h * 5 + 2.0 ** -20 / h * np.abs(f64(dy)).sum()
    assert abs((f(x + h * v, g, b) - f(x - h * v, g, b)) / (2 * h) - (f64(dx) * f64(v)).sum()) < tol
    vg = torch.randn(96, generator=gen)
    assert abs((f(x, g + h * vg, b) - f(x, g - h * vg, b)) / (2 * h) - (f64(dg) * f64(vg)).sum()) < tol
    assert abs((f(x, g, b + h * vg) - f(x, g, b - h * vg)) / (2 * h) - (f64(db) * f64(vg)).sum()) < tol
