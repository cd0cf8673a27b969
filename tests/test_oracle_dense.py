"""Pins of the FP64 oracle of the 16-bit operators: closed forms, PyTorch's own FP64 operators, and
central differences for every gradient (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import dense

RNG = np.random.default_rng


def _differences(f, a, g, h=1e-5):
    """d sum(f * g) / da by central differences, element by element."""
    d = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        p, m = a.copy(), a.copy()
        p[i] += h
        m[i] -= h
        d[i] = ((f(p) - f(m)) * g).sum() / (2 * h)
    return d


@pytest.mark.parametrize("name", dense.ACTIVATIONS)
def test_activations_and_slopes(name):
    z = np.linspace(-6, 6, 121) + 1e-3
    t = torch.from_numpy(z)
    want = {"none": t, "relu": torch.relu(t), "silu": torch.nn.functional.silu(t),
            "gelu": torch.nn.functional.gelu(t), "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}[name]
    np.testing.assert_allclose(dense.act(z, name), want.numpy(), rtol=1e-13, atol=1e-14)
    h = 1e-6
    diff = (dense.act(z + h, name) - dense.act(z - h, name)) / (2 * h)
    np.testing.assert_allclose(dense.act_slope(z, name), diff, rtol=0, atol=1e-8)


def test_grouped_mm_and_gradients():
    r = RNG(1)
    offsets = [1, 3, 3, 7]                       # an empty expert, rows before and behind the segments
    x, w, dy = r.standard_normal((8, 3)), r.standard_normal((3, 4, 3)), r.standard_normal((8, 4))
    y = dense.grouped_mm(x, w, offsets)
    np.testing.assert_allclose(y[1:3], np.einsum("mk,nk->mn", x[1:3], w[0]))
    np.testing.assert_allclose(y[3:7], np.einsum("mk,nk->mn", x[3:7], w[2]))
    assert np.isnan(y[0]).all() and np.isnan(y[7]).all()
    keep = np.zeros((8, 4))
    dx, dw = dense.grouped_mm_backward(dy, x, w, offsets, dx=np.zeros_like(x))
    np.testing.assert_allclose(dx, _differences(lambda a: dense.grouped_mm(a, w, offsets, keep), x, dy), atol=1e-8)
    np.testing.assert_allclose(dw, _differences(lambda a: dense.grouped_mm(x, a, offsets, keep), w, dy), atol=1e-8)
    assert (dw[1] == 0).all()


@pytest.mark.parametrize("name", dense.ACTIVATIONS)
def test_linear_gradients(name):
    r = RNG(2)
    x, w, b, res = (r.standard_normal(s) for s in ((5, 3), (4, 3), (4,), (5, 4)))
    dy = r.standard_normal((5, 4))
    y, z = dense.linear(x, w, b, name, res)
    np.testing.assert_allclose(y, dense.act(x @ w.T + b, name) + res)
    dx, dw, db = dense.linear_backward(dy, x, w, z, name)
    f = lambda **k: dense.linear(**{**dict(x=x, w=w, bias=b, act_name=name, residual=res), **k})[0]  # noqa: E731
    np.testing.assert_allclose(dx, _differences(lambda a: f(x=a), x, dy), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(lambda a: f(w=a), w, dy), atol=1e-7)
    np.testing.assert_allclose(db, _differences(lambda a: f(bias=a), b, dy), atol=1e-7)


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_gradients(rms):
    r = RNG(3)
    x, g, b = r.standard_normal((4, 6)) * 2 + 0.5, r.standard_normal(6), r.standard_normal(6)
    dy = r.standard_normal((4, 6))
    beta = None if rms else b
    y, mean, rstd = dense.layer_norm(x, g, beta, 1e-3, rms)
    if not rms:
        want = torch.nn.functional.layer_norm(torch.from_numpy(x), (6,), torch.from_numpy(g), torch.from_numpy(b), 1e-3)
        np.testing.assert_allclose(y, want.numpy(), rtol=1e-12)
    else:
        np.testing.assert_allclose(y, x / np.sqrt((x ** 2).mean(1, keepdims=True) + 1e-3) * g)
    dx, dg, db = dense.layer_norm_backward(dy, x, g, mean, rstd, rms)
    np.testing.assert_allclose(dx, _differences(lambda a: dense.layer_norm(a, g, beta, 1e-3, rms)[0], x, dy), atol=1e-7)
    np.testing.assert_allclose(dg, _differences(lambda a: dense.layer_norm(x, a, beta, 1e-3, rms)[0], g, dy), atol=1e-7)
    if not rms:
        np.testing.assert_allclose(db, _differences(lambda a: dense.layer_norm(x, g, a, 1e-3)[0], b, dy), atol=1e-7)
