"""Layer norm of tensors of more than 2^31 elements: sampled rows of y and dx, among them the first whose offsets pass
31 and 32 bits, and sampled columns of dgamma and dbeta, against FP64.  dy is independent of x, and the outputs hold NaN
before the calls.  Bounds as for the small shapes."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_norm import E, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()
    yield
    torch.cuda.empty_cache()


# wide rows (two passes), the widest rows of the rings, rows that start inside vectors, many narrow rows
@pytest.mark.parametrize("rows,cols,chains", [(152001, 28671, 144), (270001, 16384, 148), (480001, 9001, 144),
                                              (2300001, 1904, 8 * 148)])
def test_offsets_beyond_32_bits(rows, cols, chains):
    torch.cuda.empty_cache()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    new = lambda: torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy, out = new(), new(), new()
    for r in range(0, rows, 20000):                        # drawn in parts: no FP32 copy of the whole
        n = min(20000, rows - r)
        x[r:r + n] = torch.randn((n, cols), generator=gen, device="cuda") * 2 + 0.5
        dy[r:r + n] = torch.randn((n, cols), generator=gen, device="cuda")
    gamma, beta = 1 + 0.2 * torch.randn(cols, generator=gen, device="cuda"), torch.randn(cols, generator=gen, device="cuda")
    edges = {b // cols + d for b in (1 << 31, 1 << 32) for d in (-1, 0, 1)}
    rng = np.random.default_rng(cols)
    picks = sorted(edges | {0, 1, rows // 3, rows - 2, rows - 1} | set(rng.integers(0, rows, 8).tolist()))
    assert max(edges) < rows
    at = torch.tensor(picks, device="cuda")
    X, D, G, B = f64(x[at]), f64(dy[at]), f64(gamma), f64(beta)

    out.fill_(float("nan"))
    y, mean, rstd = moe.layer_norm(x, gamma, beta, stats=True, out=out)
    assert not torch.isnan(y.view(-1)[::97]).any() and not torch.isnan(rstd).any()
    Y, MEAN, R = dense.layer_norm(X, G, B, float(np.float32(1e-5)))
    em = 48 * E * np.abs(X).mean(1) + E * np.abs(MEAN)
    er = R * (29 * E + 0.5 * (em * R) ** 2)
    check(mean[at], MEAN, em, "mean")
    check(rstd[at], R, er, "rstd")
    rel = (er / R)[:, None] + 8 * E
    check(y[at], Y, np.abs(G) * (R * em)[:, None] * (1 + rel) + rel * np.abs(Y - B) + 2 * E * np.abs(Y), "y")

    out.fill_(float("nan"))
    dx, dg, db = moe.layer_norm_backward(dy, x, gamma, mean, rstd, dx=out)
    assert not torch.isnan(dx.view(-1)[::97]).any()
    m64, r64 = f64(mean[at]), f64(rstd[at])
    DX, _, _ = dense.layer_norm_backward(D, X, G, m64, r64)
    XH, GG = (X - m64[:, None]) * r64[:, None], D * G
    eg = 4 * np.abs(GG) + 52 * np.abs(GG).mean(1, keepdims=True) + \
        np.abs(XH) * 58 * np.abs(GG * XH).mean(1, keepdims=True)
    check(dx[at], DX, r64[:, None] * E * eg, "dx")
    assert np.abs(DX).max() > 0.1
    for c in [0, 1, cols // 2, cols - 1] + rng.integers(0, cols, 4).tolist():
        d, xh = dy[:, c].double(), (x[:, c].double() - mean.double()) * rstd.double()
        bound = lambda t: (rows + 8) * E * np.array([float(t.abs().sum())])  # noqa: E731
        check(dg[c:c + 1], np.array([float((d * xh).sum())]), bound(d * xh), ("dgamma", c))
        check(db[c:c + 1], np.array([float(d.sum())]), bound(d), ("dbeta", c))
        # The terms have both signs and a spread of about 1, so a chain of n additions stays below 6 sqrt(n) and its
        # roundings add up to n E 6 sqrt(n) at most; over all chains (one a group of threads) that is
        # rows E 6 sqrt(rows / chains), less than 0.05 sqrt(rows) here.  Sums over wrong rows would differ by about sqrt(rows).
        assert rows * E * 6 / chains ** 0.5 < 0.05
        assert abs(float(dg[c]) - float((d * xh).sum())) < 0.05 * rows ** 0.5
        assert abs(float(db[c]) - float(d.sum())) < 0.05 * rows ** 0.5
