"""Pins of oracle.dense: hand-worked values and gradients against central
differences of the forward definitions."""

import math

import numpy as np
import pytest

from oracle import dense as od

KINDS = ("none", "silu", "gelu", "relu")


def _differences(f, a, rng, n=12, step=1e-6):
    """(index, central difference of the scalar f along a's element) samples."""
    for _ in range(n):
        i = tuple(rng.integers(0, s) for s in a.shape)
        hi, lo = a.copy(), a.copy()
        hi[i] += step
        lo[i] -= step
        yield i, (f(hi) - f(lo)) / (2 * step)


def test_activations_at_known_points():
    assert od.act("silu", [0.0, math.log(3.0)]).tolist() == pytest.approx([0.0, 0.75 * math.log(3.0)], abs=1e-15)
    # Phi(1) = 0.8413447460685429
    assert od.act("gelu", [1.0])[0] == pytest.approx(0.8413447460685429, abs=1e-15)
    assert od.act("relu", [-2.0, 0.0, 3.0]).tolist() == [0.0, 0.0, 3.0]
    assert od.act_grad("relu", [-2.0, 0.0, 3.0]).tolist() == [0.0, 0.0, 1.0]
    z = np.linspace(-6, 6, 41) + 0.01          # off the corner of relu
    for k in KINDS:
        num = (od.act(k, z + 1e-6) - od.act(k, z - 1e-6)) / 2e-6
        assert np.allclose(od.act_grad(k, z), num, atol=1e-8), k


def test_gelu_tail():
    # Phi(-8), Phi(-12) from tables of the normal distribution
    for z, phi in ((-8.0, 6.22096057427178e-16), (-12.0, 1.776482112077679e-33)):
        pdf = math.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        assert od.act("gelu", [z])[0] == pytest.approx(z * phi, rel=1e-12, abs=0)
        assert od.act_grad("gelu", [z])[0] == pytest.approx(phi + z * pdf, rel=1e-12, abs=0)


def test_layer_norm_by_hand():
    # deviations -1, 1 around 3: var 1, eps 3 -> rstd 1/2
    y, mean, rstd, s = od.layer_norm([[1.0, 3.0]], gamma=[2.0, 4.0], beta=[0.5, -0.5], eps=3.0, residual=[[1.0, 1.0]])
    assert mean.tolist() == [3.0] and rstd.tolist() == [0.5]
    assert s.tolist() == [[2.0, 4.0]]
    assert y.tolist() == [[-0.5, 1.5]]


@pytest.mark.parametrize("with_gamma", [False, True])
def test_layer_norm_gradient_is_the_forward_s(with_gamma):
    r = np.random.default_rng(0)
    x, dy, dsum = r.standard_normal((3, 7)) * 2 + 1, r.standard_normal((3, 7)), r.standard_normal((3, 7))
    gamma = r.standard_normal(7) if with_gamma else None
    beta = r.standard_normal(7)

    def loss(x=x, gamma=gamma, beta=beta):
        y, _, _, s = od.layer_norm(x, gamma, beta)
        return float((y * dy).sum() + (s * dsum).sum())

    _, mean, rstd, s = od.layer_norm(x, gamma, beta)
    dx, dgamma, dbeta = od.layer_norm_backward(dy, s, mean, rstd, gamma, dsum)
    for i, d in _differences(lambda v: loss(x=v), x, r):
        assert dx[i] == pytest.approx(d, abs=1e-7)
    if with_gamma:
        for i, d in _differences(lambda v: loss(gamma=v), gamma, r):
            assert dgamma[i] == pytest.approx(d, abs=1e-7)
    for i, d in _differences(lambda v: loss(beta=v), beta, r):
        assert dbeta[i] == pytest.approx(d, abs=1e-7)


@pytest.mark.parametrize("kind", KINDS)
def test_linear_gradient_is_the_forward_s(kind):
    r = np.random.default_rng(1)
    x, w, b = r.standard_normal((4, 5)), r.standard_normal((6, 5)), r.standard_normal(6)
    res, dy = r.standard_normal((4, 6)), r.standard_normal((4, 6))

    def loss(x=x, w=w, b=b):
        return float((od.linear(x, w, b, kind, res)[0] * dy).sum())

    z = od.linear(x, w, b, kind, res)[1]
    dx, dw, db, _ = od.linear_backward(dy, x, w, z, kind)
    for got, arr, name in ((dx, x, "x"), (dw, w, "w"), (db, b, "b")):
        for i, d in _differences(lambda v: loss(**{name: v}), arr, r):
            assert got[i] == pytest.approx(d, abs=1e-6), name


@pytest.mark.parametrize("kind", KINDS)
def test_gated_gradient_is_the_forward_s(kind):
    r = np.random.default_rng(2)
    x, w13, da = r.standard_normal((4, 5)), r.standard_normal((6, 5)), r.standard_normal((4, 3))

    def loss(x=x, w13=w13):
        return float((od.gated_linear(x, w13, kind)[0] * da).sum())

    h = od.gated_linear(x, w13, kind)[1]
    dx, dw, _ = od.gated_linear_backward(da, x, w13, h, kind)
    for got, arr, name in ((dx, x, "x"), (dw, w13, "w13")):
        for i, d in _differences(lambda v: loss(**{name: v}), arr, r):
            assert got[i] == pytest.approx(d, abs=1e-6), name


def test_gate_rows_come_first():
    # one token, I = 1: g = 2, u = 3
    a, h = od.gated_linear([[1.0]], [[2.0], [3.0]], "relu")
    assert h.tolist() == [[2.0, 3.0]] and a.tolist() == [[6.0]]
    a, _ = od.gated_linear([[1.0]], [[-2.0], [3.0]], "relu")
    assert a.tolist() == [[0.0]]
