"""Pins of oracle.experts: hand-worked values, gradients against central
differences of the forward definitions, the whole pass against its parts."""

import numpy as np
import pytest

from oracle import experts as oe

OFF = [0, 2, 2, 5]
ROWS = [3, 0, 1, 1, 2]


def _inputs(seed=0):
    r = np.random.default_rng(seed)
    return r, r.standard_normal((4, 3)), r.standard_normal((3, 6, 3)), r.random(5) + 0.5


def test_grouped_linear_by_hand():
    x = [[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]
    w = [[[1.0, 0.0]], [[0.0, 10.0]]]
    assert oe.grouped_linear(x, w, [0, 1, 3]).tolist() == [[1.0], [40.0], [60.0]]
    # by index, one outside the source; a row behind the last group
    y = oe.grouped_linear(x, w, [0, 1, 3], [2, 7, 0, 1])
    assert y[:3].tolist() == [[5.0], [0.0], [20.0]] and np.isnan(y[3]).all()


def test_empty_group_has_no_weight_gradient():
    r, x, w, _ = _inputs()
    dy = r.standard_normal((5, 6))
    dx, dw = oe.grouped_linear_backward(dy, x, w, OFF, ROWS)
    assert not dw[1].any() and dw[0].any() and dx.shape == (5, 3)


def _check(f, a, grad, r):
    for _ in range(10):
        i = tuple(r.integers(0, s) for s in a.shape)
        hi, lo = a.copy(), a.copy()
        hi[i] += 1e-6
        lo[i] -= 1e-6
        assert grad[i] == pytest.approx((f(hi) - f(lo)) / 2e-6, rel=1e-6, abs=1e-7), i


def test_grouped_linear_gradients():
    r, x, w, _ = _inputs(1)
    src = r.standard_normal((4, 6))
    dy_rows = [0, 3, 2, 2, 1]
    dx, dw = oe.grouped_linear_backward(src, x, w, OFF, ROWS, dy_rows)
    dy = oe.take(src, dy_rows)
    _check(lambda a: (oe.grouped_linear(x, a, OFF, ROWS) * dy).sum(), w, dw, r)
    # dx per row: the gradient of the gathered rows
    xr = oe.take(x, ROWS)
    _check(lambda a: (oe.grouped_linear(a, w, OFF) * dy).sum(), xr, dx, r)


@pytest.mark.parametrize("kind", ["silu", "gelu", "none"])
def test_gated_gradients(kind):
    r, x, w13, s = _inputs(2)
    da = r.standard_normal((5, 3))
    xr = oe.take(x, ROWS)
    _, h = oe.grouped_gated_linear(x, w13, OFF, kind, ROWS, s)
    dx, dw, ds, dh = oe.grouped_gated_linear_backward(da, x, w13, h, OFF, kind, ROWS, s)
    _check(lambda a: (oe.grouped_gated_linear(x, a, OFF, kind, ROWS, s)[0] * da).sum(), w13, dw, r)
    _check(lambda a: (oe.grouped_gated_linear(a, w13, OFF, kind, None, s)[0] * da).sum(), xr, dx, r)
    _check(lambda a: (oe.grouped_gated_linear(x, w13, OFF, kind, ROWS, a)[0] * da).sum(), s, ds, r)
    assert dh.shape == h.shape


def test_quant_int8_by_hand():
    q, s = oe.quant_int8([[127.0, -63.5, 0.5, 1.5, -2.5], [0.0] * 5, [-254.0, 1.0, 3.0, 0.0, 254.0]])
    assert s.tolist() == [1.0, 1.0, 2.0]
    assert q.tolist() == [[127, -64, 0, 2, -2], [0] * 5, [-127, 0, 2, 0, 127]]     # ties to even
    # the smallest magnitudes: max / 127 rounds to no float above 0, or to one too small
    tiny = np.float32(2.0 ** -149)
    q, s = oe.quant_int8(np.array([[tiny, 0], [190 * tiny, -190 * tiny]], np.float32))
    assert s.tolist() == [1.0, float(tiny)] and q.tolist() == [[0, 0], [127, -127]]
    q, s = oe.quant_int8(np.array([[1.0, np.nan], [np.inf, 2.0]], np.float32))
    assert np.isnan(s).all() and not q.any()


def test_int8_linear_by_hand():
    y, total = oe.int8_linear([[1.0, 2.0], [-3.0, 4.0]], [0.5, 2.0], [[[10.0, 1.0]], [[1.0, 1.0]]], [[3.0], [1.0]],
                              [0, 1, 2], [1, 0])
    assert total.tolist() == [[-26.0], [3.0]] and y.tolist() == [[-156.0], [1.5]]


def test_router_gradient_is_the_gates():
    r = np.random.default_rng(3)
    z, d = r.standard_normal((4, 6)), r.standard_normal((4, 2))
    top = np.array([[0, 5], [2, 1], [3, 4], [5, 0]])

    def loss(z):
        s = 1.0 / (1.0 + np.exp(-np.take_along_axis(z, top, 1)))
        return (s / s.sum(1, keepdims=True) * d).sum()

    _check(loss, z, oe.router_backward(d, top, z), r)


def test_whole_pass_is_its_parts():
    r = np.random.default_rng(4)
    T, E, K, H, I = 5, 3, 2, 4, 3
    x, w13, w2 = r.standard_normal((T, H)), r.standard_normal((E + 1, 2 * I, H)), r.standard_normal((E + 1, H, I))
    top = np.array([r.permutation(E)[:K] for _ in range(T)])
    gates = r.random((T, K))
    # rows by expert, the shared expert's last
    order = sorted((int(top[t, k]), t, k) for t in range(T) for k in range(K))
    off = np.searchsorted([e for e, _, _ in order], range(E + 1)).tolist() + [T * K + T]
    rows = [t for _, t, _ in order] + list(range(T))
    scale = [gates[t, k] for _, t, k in order] + [1.0] * T
    a, _ = oe.grouped_gated_linear(x, w13, off, "silu", rows, scale)
    o = oe.grouped_linear(a, w2, off)
    y = np.zeros((T, H))
    np.add.at(y, rows, o)
    assert np.allclose(y, oe.moe_ffn(x, w13[:E], w2[:E], top, gates, shared=(w13[E], w2[E])), atol=1e-12)
