"""The experts' passes with float32 results: the terms of the sums over a token's experts are not rounded on the way."""

import numpy as np
import pytest
import torch

from gpu_util import banner, host
from oracle import experts as oe
from test_gpu_dense import U, V, _close, _mat, _norms
from test_gpu_experts import _layer, _per_row

pytestmark = pytest.mark.gpu
T, H, I, E, K = 200, 136, 72, 7, 3
F32 = torch.float32


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _sum(rows, tokens):
    out = np.zeros((T, rows.shape[1]))
    np.add.at(out, tokens, rows)
    return out


@pytest.mark.parametrize("n_shared", [0, 1])
def test_bf16_pass_with_float32_results(d, n_shared):
    banner(f"moe_ffn with float32 results, shared {n_shared}")
    r = np.random.default_rng(21)
    x, x64, w13, w13_64, w2, w2_64, logits, routing = _layer(d, r, T, H, I, E, K, n_shared, 0.15)
    y, saved = d.moe_ffn_forward(x, routing, w13, w2, n_shared=n_shared, training=True, out_dtype=F32)
    assert y.dtype == F32
    off, perm = host(saved["offsets"]), host(saved["perm"])
    # from the activations that it saved: a product of bf16 values, K + 1 terms summed in float32
    a64 = host(saved["a"]).astype(np.float64)
    o = oe.grouped_linear(a64, w2_64, off)
    terms = _per_row(off, perm.size, lambda g, p: _norms(a64[p], w2_64[g]), H)
    _close(y, _sum(o, perm), 16 * U * _sum(terms, perm) + (K + 1) * U * _sum(np.abs(o), perm), "f32", "y")
    y16, _ = d.moe_ffn_forward(x, routing, w13, w2, n_shared=n_shared)
    assert y16.dtype == torch.bfloat16 and not torch.equal(y16, y.bfloat16())     # the default rounds the terms
    dy, _ = _mat(r, T, H, 0.1)
    got = d.moe_ffn_backward(dy, x, routing, w13, w2, saved, logits=logits, dx_dtype=F32)
    assert got["dx"].dtype == F32
    da, _ = d.grouped_linear_backward(dy, saved["a"], w2, saved["offsets"], dy_rows=saved["perm"])
    dz = oe.grouped_gated_linear_backward(host(da).astype(np.float64), oe.take(x64, perm), w13_64,
                                          host(saved["h"]).astype(np.float64), off, "silu", None,
                                          host(saved["scale"]).astype(np.float64))[3]
    rows = _per_row(off, perm.size, lambda g, p: dz[p] @ w13_64[g], H)
    # dh as two bf16 values, as float32 gradients take it
    bound = _per_row(off, perm.size, lambda g, p: 16 * U * _norms(dz[p], w13_64[g].T) +
                     (4 * V * V + 2.0 ** -19) * np.sqrt((dz[p] ** 2) @ (w13_64[g] ** 2)), H)
    _close(got["dx"], _sum(rows, perm), _sum(bound, perm) + (K + 1) * U * _sum(np.abs(rows), perm), "f32", "dx")
    other = d.moe_ffn_backward(dy, x, routing, w13, w2, saved, logits=logits)
    assert other["dx"].dtype == torch.bfloat16
    assert all(torch.equal(got[k], other[k]) for k in ("dw13", "dw2", "dgates", "dlogits"))


@pytest.mark.parametrize("n_shared", [0, 1])
def test_8_bit_pass_with_float32_results(d, n_shared):
    banner(f"moe_ffn int8 with float32 results, shared {n_shared}")
    r = np.random.default_rng(22)
    x, _, w13, _, w2, _, _, routing = _layer(d, r, T, H, I, E, K, n_shared)
    q13, q2 = d.quant_rows_int8(w13), d.quant_rows_int8(w2)
    y = d.moe_ffn_int8_forward(x, routing, q13, q2, n_shared=n_shared, out_dtype=F32)
    assert y.dtype == F32
    off, perm, scale, _ = d.experts._routed_rows(routing, n_shared)
    a = d.int8_gated_linear(*d.quant_rows_int8(x), *q13, off, rows=perm, row_scale=scale)
    q, s = (host(t).astype(np.float64) for t in d.quant_rows_int8(a))
    o, _ = oe.int8_linear(q, s, host(q2[0]).astype(np.float64), host(q2[1]).astype(np.float64), host(off))
    tokens = host(perm)
    # exact sums rounded once and multiplied twice, then the sum over the experts
    _close(y, _sum(o, tokens), (3.01 + K + 1) * U * _sum(np.abs(o), tokens), "f32", "y")
