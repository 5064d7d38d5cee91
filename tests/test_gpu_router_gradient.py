"""The router logits' gradient, of dsmoe_router_backward and dsmoe_gate_backward,
where a sigmoid saturates and where the chosen ones are tiny.

Bound: the formula in double, of K sums, is within (8 K + 32) 2^-53 of the size of
its terms, sum_j |d_k - d_j| gate_j gate_k (1 - s_k); it is rounded to float32 once,
2^-24 of the value or half a step of the smallest numbers, 2^-150.
"""

import numpy as np
import pytest
import torch

from gpu_util import banner, dev, host
from oracle import backward as ob
from oracle import experts as oe
from test_gpu_dense import _close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _bound(dg, top, z):
    T, K = top.shape
    zs = np.take_along_axis(z.astype(np.float64), top.astype(np.int64), 1)
    s, q = 1 / (1 + np.exp(-zs)), 1 / (1 + np.exp(zs))
    gate = s / s.sum(1, keepdims=True)
    terms = np.einsum("tkj,tj->tk", np.abs(dg[:, :, None] - dg[:, None, :].astype(np.float64)), gate) * gate * q
    out = np.zeros(z.shape)
    np.add.at(out, (np.arange(T)[:, None], top), (8 * K + 32) * 2.0 ** -53 * terms + 2.0 ** -150)
    return out


def _logits(r, T, E, lo, hi, signs):
    """Magnitudes in [lo, hi] with one of the signs for each token."""
    z = r.uniform(lo, hi, (T, E)) * r.choice(signs, (T, 1))
    return z.astype(np.float32)


# the derivative of a sigmoid past float32's 1 - s, sums of tiny sigmoids, both in one token
RANGES = [(10, 17, (1,)), (17, 30, (1,)), (60, 85, (1,)), (10, 30, (-1,)), (80, 100, (-1,)), (0, 30, (-1, 1)), (-30, 30, (1,))]


@pytest.mark.parametrize("lo,hi,signs", RANGES)
@pytest.mark.parametrize("T,E,K", [(1, 4, 1), (1, 4, 2), (50, 64, 8), (7, 1024, 32)])
def test_router_backward_keeps_its_digits(d, T, E, K, lo, hi, signs):
    banner(f"router_backward {T} {E} {K}, logits {lo} to {hi} times {signs}")
    r = np.random.default_rng(T + K)
    z = _logits(r, T, E, lo, hi, signs)
    top = np.stack([r.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    dg = r.standard_normal((T, K)).astype(np.float32)
    got = d.router_backward(dev(dg), dev(top), dev(z))
    _close(got, oe.router_backward(dg, top, z), _bound(dg, top, z), "f32", "dlogits")
    if K > 1:
        assert (host(got) != 0).sum() >= T * (K - 1), "gradients that float32 holds"


@pytest.mark.parametrize("lo,hi,signs", RANGES)
@pytest.mark.parametrize("T,E,K,H", [(3, 8, 2, 64), (40, 64, 8, 256), (2, 1024, 32, 8)])
def test_gate_backward_keeps_its_digits(d, T, E, K, H, lo, hi, signs):
    banner(f"gate_backward {T} {E} {K}, logits {lo} to {hi} times {signs}")
    r = np.random.default_rng(T + K)
    z = _logits(r, T, E, lo, hi, signs)
    top = np.stack([r.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    inv = r.permutation(T * K).astype(np.int32).reshape(T, K)
    dy, o = (dev(r.standard_normal(s).astype(np.float32), torch.bfloat16) for s in ((T, H), (T * K, H)))
    dgate, dz = d.gate_backward(dy, o, dev(inv), dev(top), dev(z))
    # the gates' gradients have a test of their own: theirs are this formula's input
    dg = host(dgate).astype(np.float64)
    want, want_z = ob.gate_backward(host(dy), host(o)[inv], top, z, E)
    assert np.abs(dg - want).max() <= 1e-5 * H
    _close(dz, oe.router_backward(dg, top, z), _bound(dg, top, z), "f32", "dlogits")
    assert np.allclose(want_z, oe.router_backward(want, top, z), rtol=1e-6, atol=0)


def test_an_expert_chosen_twice_and_indices_outside(d):
    """The gradients of an expert's choices add up, in either call; dsmoe_router_backward leaves indices outside [0, E)
    out."""
    banner("router gradient, an expert chosen twice")
    r = np.random.default_rng(5)
    T, E, K, H = 20, 70, 6, 64
    z = r.standard_normal((T, E)).astype(np.float32)
    top = np.stack([r.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    top[:, 3], top[::2, 5] = top[:, 0], top[::2, 0]
    dg = r.standard_normal((T, K)).astype(np.float32)
    # three roundings to float32 and two sums of them at most
    size = np.zeros((T, E))
    np.add.at(size, (np.arange(T)[:, None], top), np.abs(dg).max(1, keepdims=True) * 2.0 ** -22)
    _close(d.router_backward(dev(dg), dev(top), dev(z)), oe.router_backward(dg, top, z), size, "f32", "router_backward")
    inv = r.permutation(T * K).astype(np.int32).reshape(T, K)
    dy, o = (dev(r.standard_normal(s).astype(np.float32), torch.bfloat16) for s in ((T, H), (T * K, H)))
    dgate, dz = d.gate_backward(dy, o, dev(inv), dev(top), dev(z))
    dg2 = host(dgate).astype(np.float64)
    size2 = size / np.abs(dg).max(1, keepdims=True) * np.abs(dg2).max(1, keepdims=True)
    _close(dz, oe.router_backward(dg2, top, z), size2, "f32", "gate_backward")
    out = top.copy()
    out[:, 0], out[:, 2] = -1, E
    left = [1, 3, 4, 5]
    _close(d.router_backward(dev(dg), dev(out), dev(z)), oe.router_backward(dg[:, left], out[:, left], z), size, "f32",
           "indices outside")
