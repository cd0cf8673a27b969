"""The 16-bit operators around the quantised layer in FP64: products grouped by expert, the dense
product with its epilogue, the layer norm, and their gradients.  TEST INFRASTRUCTURE ONLY.

Plain formulas on FP64 arrays; nothing is rounded (a test rounds the operands it hands to the
kernels first and bounds the kernels' own roundings).
"""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_erf = np.vectorize(math.erf, otypes=[np.float64])
_C = math.sqrt(2.0 / math.pi)


def act(z, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    return z


def act_slope(z, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def segments(offsets):
    """(expert, slice of rows) of every segment."""
    return [(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(len(offsets) - 1)]


def grouped_mm(x, w, offsets, out=None):
    """y[i] = x[i] w[e]^T; rows outside the segments keep ``out``'s values (NaN without one)."""
    y = np.full((x.shape[0], w.shape[1]), np.nan) if out is None else np.array(out, dtype=np.float64)
    for e, rows in segments(offsets):
        y[rows] = x[rows] @ w[e].T
    return y


def grouped_mm_backward(dy, x, w, offsets, dx=None):
    dx = np.full(x.shape, np.nan) if dx is None else np.array(dx, dtype=np.float64)
    dw = np.zeros(w.shape)
    for e, rows in segments(offsets):
        dx[rows] = dy[rows] @ w[e]
        dw[e] = dy[rows].T @ x[rows]
    return dx, dw


def linear(x, w, bias=None, act_name="none", residual=None):
    """(y, z)"""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, act_name)
    return (y if residual is None else y + residual), z


def linear_backward(dy, x, w, z=None, act_name="none"):
    """(dx, dw, db)"""
    dz = dy if act_name == "none" else dy * act_slope(z, act_name)
    return dz @ w, dz.T @ x, dz.sum(0)


def layer_norm(x, gamma=None, beta=None, eps=1e-5, rms=False):
    """(y, mean, rstd); mean is zero with rms."""
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, rms=False):
    """(dx, dgamma, dbeta)"""
    xh = (x if rms else x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = g - xh * (g * xh).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * xh).sum(0), dy.sum(0)
