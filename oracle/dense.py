"""Dense feed-forward operators in float64: layer norm, linear with an
epilogue and gated linear, each with its gradients, from their definitions.

    layer_norm    y = (s - mean(s)) / sqrt(var(s) + eps) * gamma + beta
    linear        z = x W^T + bias,  y = act(z) + residual
    gated_linear  [g | u] = x W13^T,  a = act(g) * u

Everything is float64 (inputs are converted first); the bf16 roundings of an
implementation are its own affair and belong to the tests' bounds.
"""

import math

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def _normal_cdf(z):
    """By erfc, which keeps its digits where the value is near 0."""
    return np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in np.ravel(z)], np.float64).reshape(np.shape(z))


def act(kind, z):
    z = _f64(z)
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return z * _normal_cdf(z)
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    raise ValueError(kind)


def act_grad(kind, z):
    z = _f64(z)
    if kind == "none":
        return np.ones_like(z)
    if kind == "silu":
        sig = 1.0 / (1.0 + np.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    if kind == "gelu":
        return _normal_cdf(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    raise ValueError(kind)


def layer_norm(x, gamma=None, beta=None, eps=1e-5, residual=None):
    """(y, mean, rstd, s) with s = x + residual."""
    s = _f64(x) if residual is None else _f64(x) + _f64(residual)
    mean = s.mean(axis=1)
    d = s - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * _f64(gamma)
    if beta is not None:
        y = y + _f64(beta)
    return y, mean, rstd, s


def layer_norm_backward(dy, x, mean, rstd, gamma=None, dsum=None):
    """(dx, dgamma, dbeta) at the given statistics of x."""
    dy, x, rstd = _f64(dy), _f64(x), _f64(rstd)[:, None]
    n = (x - _f64(mean)[:, None]) * rstd
    g = dy if gamma is None else dy * _f64(gamma)
    dx = rstd * (g - g.mean(axis=1, keepdims=True) - n * (g * n).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + _f64(dsum)
    return dx, (dy * n).sum(axis=0), dy.sum(axis=0)


def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z)."""
    z = _f64(x) @ _f64(w).T
    if bias is not None:
        z = z + _f64(bias)
    y = act(kind, z)
    if residual is not None:
        y = y + _f64(residual)
    return y, z


def linear_backward(dy, x, w, z=None, kind="none"):
    """(dx, dw, dbias, dz)."""
    dz = _f64(dy) if kind == "none" else _f64(dy) * act_grad(kind, z)
    return dz @ _f64(w), dz.T @ _f64(x), dz.sum(axis=0), dz


def gated_linear(x, w13, kind="silu"):
    """(a, h)."""
    h = _f64(x) @ _f64(w13).T
    i = h.shape[1] // 2
    return act(kind, h[:, :i]) * h[:, i:], h


def gated_linear_backward(da, x, w13, h, kind="silu"):
    """(dx, dw13, dh)."""
    h, da = _f64(h), _f64(da)
    i = h.shape[1] // 2
    g, u = h[:, :i], h[:, i:]
    dh = np.concatenate([da * u * act_grad(kind, g), da * act(kind, g)], axis=1)
    return dh @ _f64(w13), dh.T @ _f64(x), dh
