"""Float32 gradients of the grouped gated product, whose second product is added to the first, in every tile that
takes them, and tiles of every height at its limits, against float64."""

import numpy as np
import pytest
import torch

import grouped_kernels as gk
from gpu_util import banner, host
from oracle import dense as od
from oracle import experts as oe
from test_gpu_dense import U, V, _mat, _vec
from test_gpu_experts import (_check_rows, _codes, _experts, _gated_check, _grad_check, _i32, _linear_bound, _nan,
                              _offsets, _scales)

pytestmark = pytest.mark.gpu

# last tiles of every height on both sides of its limit, alone and behind whole tiles
LONG = [128, 129, 192, 193, 256, 257, 320, 384, 385, 448, 449, 512, 64, 1, 0, 255] * 3
SHORT = [128, 129, 192, 193, 64, 1, 0, 127] * 6


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


@pytest.mark.parametrize("sizes,N,K,shape", [(LONG, 520, 520, "256x256"), (LONG, 522, 521, "256x256"), (SHORT, 520, 520, "128x128"),
                                             (SHORT, 264, 301, "64x64"), (SHORT, 72, 72, "32x128")])
def test_float32_dx_of_the_gated_product(d, sizes, N, K, shape):
    """N = 2 I; odd K: x and the weights are copied, once for both products."""
    R, G = sum(sizes), len(sizes)
    assert gk.shape(d.lib, "dx", G, R, N, K) == shape
    banner(f"float32 dx in {shape}: {G} groups {R} rows {N}x{K}")
    r = np.random.default_rng(N + K)
    off, doff = _offsets(sizes)
    w, w64 = _experts(r, G, N, K)
    x, x64 = _mat(r, R, K)
    h, h64 = _mat(r, R, N, 1.5)
    da, da64 = _mat(r, R, N // 2, 0.1)
    s, s64 = _vec(r, R, 0.3, 1.0)
    dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off, "silu", None, s64)[3]
    for t, rounded in (("f32", 4 * V * V + 2.0 ** -19), ("bf16", 4 * V + 2.0 ** -19)):
        dx, none, _ = d.grouped_gated_linear_backward(da, x, w, h, doff, "silu", None, s, dx=_nan(R, K, t, pad=3), need_dw=False)
        assert none is None
        _grad_check(dx, None, dz, x64, w64, off, rounded, t, None, t)
    # both gradients, each in two products with copies of its own
    dx, dw, _ = d.grouped_gated_linear_backward(da, x, w, h, doff, "silu", None, s, torch.float32, torch.float32)
    _grad_check(dx, dw, dz, x64, w64, off, 4 * V * V + 2.0 ** -19, "f32", "f32", "both")


@pytest.mark.parametrize("product,N,K,shape", [("y", 1040, 520, "256x256 each"), ("int8", 1040, 520, "256x256 each"),
                                               ("gated", 520, 520, "256x256"), ("int8 gated", 520, 520, "256x256")])
def test_tiles_of_every_height(d, product, N, K, shape):
    R, G = sum(SHORT), len(SHORT)
    assert gk.shape(d.lib, product, G, R, N, K) == shape
    banner(f"{product}: tiles of every height, {G} groups {R} rows {N}x{K}")
    r = np.random.default_rng(N)
    off, doff = _offsets(SHORT)
    n, rows = R // 2, r.integers(0, R // 2, R)
    s, s64 = _vec(r, R, 0.3, 1.0)
    if product == "y" or product == "gated":
        x, x64 = _mat(r, n, K)
        x64 = oe.take(x64, rows)
        w, w64 = _experts(r, G, N if product == "y" else 2 * N, K)
        if product == "y":
            y = d.grouped_linear(x, w, doff, _i32(rows), y=_nan(R, N))
            _check_rows(y, oe.grouped_linear(x64, w64, off), _linear_bound(x64, w64, off), off, "bf16", "y")
        else:
            a, h = d.grouped_gated_linear(x, w, doff, "silu", _i32(rows), s, a=_nan(R, N), save_h=True)
            _gated_check(a, h, x64, w64, s64, off, "silu", "bf16", "gated")
        return
    x, x64 = _codes(r, n, K)
    w, w64 = _codes(r, G, N if product == "int8" else 2 * N, K)
    (xs, xs64), (ws, _) = _scales(r, n), _scales(r, G, w.shape[1])
    ws = ws / K
    want, _ = oe.int8_linear(x64, xs64, w64, host(ws).astype(np.float64), off, rows)
    if product == "int8":
        y = d.int8_linear(x, xs, w, ws, doff, _i32(rows), y=_nan(R, N))
        _check_rows(y, want, 3.01 * U * np.abs(want), off, "bf16", "y")
        return
    a = d.int8_gated_linear(x, xs, w, ws, doff, "silu", _i32(rows), s, a=_nan(R, N))
    g, u = want[:, :N], want[:, N:]
    f, hb = np.abs(od.act("silu", g)), 3.01 * U * np.abs(want)
    bound = np.abs(s64)[:, None] * (1.13 * hb[:, :N] * (np.abs(u) + hb[:, N:]) + f * hb[:, N:] +
                                    (2.0 ** -20 + 2 * U) * f * np.abs(u))
    _check_rows(a, s64[:, None] * od.act("silu", g) * u, bound, off, "bf16", "a")
