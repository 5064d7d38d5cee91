"""The oracle's router gradient against closed forms where a sigmoid is near 0 or 1."""

import numpy as np
import pytest

from oracle import backward as ob
from oracle import experts as oe


@pytest.mark.parametrize("z", [0.0, 9.0, 17.5, 30.0, 45.0, 100.0, -9.0, -30.0, -100.0])
def test_equal_logits(z):
    """K equal logits: the gates are 1 / K, so the gradient is (d_k - mean d) (1 - s) / K, and 1 - s is
    e^-z / (1 + e^-z)."""
    r = np.random.default_rng(3)
    T, E, K, H = 4, 8, 4, 16
    top = np.stack([r.permutation(E)[:K] for _ in range(T)])
    logits = np.full((T, E), z, np.float32)
    q = np.exp(-z) / (1 + np.exp(-z)) if z > 0 else 1 / (1 + np.exp(z))
    dy, o = r.standard_normal((T, H)), r.standard_normal((T, K, H))
    d, dz = ob.gate_backward(dy, o, top, logits, E)
    want = np.zeros((T, E))
    np.put_along_axis(want, top, (d - d.mean(1, keepdims=True)) * q / K, 1)
    assert np.allclose(dz, want, rtol=1e-12, atol=0)
    assert np.allclose(oe.router_backward(d, top, logits), want, rtol=1e-12, atol=0)


def test_two_logits_far_apart():
    """gate_0 = s_0 / (s_0 + s_1): with d = (1, 0) the gradients are gate_0 gate_1 (1 - s_k), the second's negative."""
    z = np.array([[20.0, -25.0]], np.float32)
    s, q = 1 / (1 + np.exp(-z.astype(np.float64))), 1 / (1 + np.exp(z.astype(np.float64)))
    g = s / s.sum()
    want = g[0, 0] * g[0, 1] * q * [1, -1]
    got = oe.router_backward(np.array([[1.0, 0.0]]), np.array([[0, 1]]), z)
    assert np.allclose(got, want, rtol=1e-12, atol=0)


def test_an_expert_chosen_twice():
    """Its logit moves both of its gates: the gradient is the sum, as differences give it."""
    z, d = np.array([[0.3, -1.2, 2.0]]), np.array([[0.7, -0.4, 1.1]])
    top = np.array([[2, 0, 2]])

    def loss(z):
        s = 1 / (1 + np.exp(-z[0, top[0]]))
        return float((d[0] * s / s.sum()).sum())

    num = [(loss(z + e) - loss(z - e)) / 2e-6 for e in 1e-6 * np.eye(3)]
    assert np.allclose(oe.router_backward(d, top, z)[0], num, atol=1e-8)
    _, dz = ob.gate_backward(np.ones((1, 1)), d[:, :, None], top, z, 3)    # z in float32 there
    assert np.allclose(dz[0], num, atol=1e-6)
