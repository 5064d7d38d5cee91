"""Float32 gradients whose upstream gradient enters as two bf16 values, where the other operand holds an infinity: an
infinity of the product's sign, as in the formula, and not the NaN of the second value's product."""

import numpy as np
import pytest
import torch

from gpu_util import banner
from oracle import dense as od
from oracle import experts as oe
from test_gpu_dense import V, _mat
from test_gpu_dense import _grad_check as _dense_check
from test_gpu_experts import _experts, _grad_check, _offsets

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _signs(got, want, what):
    """Infinities with want's signs (want is nowhere 0)."""
    assert torch.isinf(got).all(), (what, int(torch.isnan(got).sum()), "NaN")
    assert torch.equal(got > 0, torch.from_numpy(want > 0).cuda()), what


# small tiles, and dx by a block for each 256-row tile with dw by blocks that stay
@pytest.mark.parametrize("sizes,I,H", [([30, 0, 41, 9], 36, 72), ([300, 129, 420, 300] * 10, 260, 520)])
def test_grouped_gated_linear_backward(d, sizes, I, H):
    banner(f"infinite x and w: {len(sizes)} groups, {I}x{H}")
    R, G = sum(sizes), len(sizes)
    r = np.random.default_rng(I)
    off, doff = _offsets(sizes)
    w, w64 = _experts(r, G, 2 * I, H)
    x, x64 = _mat(r, R, H)
    h, h64 = _mat(r, R, 2 * I, 1.5)
    da, da64 = _mat(r, R, I, 0.1)
    dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off, "silu")[3]
    row, group = off[2] + 5, 2
    x[row, 7] = float("inf")
    w[group, 3, 11] = -float("inf")
    dx, dw, _ = d.grouped_gated_linear_backward(da, x, w, h, doff, dx_dtype=F32, dw_dtype=F32)
    mine = slice(off[2], off[3])
    _signs(dw[group, :, 7], dz[row], "dw")
    _signs(dx[mine, 11], -dz[mine, 3], "dx")
    # everything else as without them
    dx[mine, 11], dw[group, :, 7] = 0, 0
    wx, ww = w64.copy(), x64.copy()
    wx[group, :, 11], ww[mine, 7] = 0, 0
    bound = 4 * V * V + 2.0 ** -19
    _grad_check(dx, None, dz, x64, wx, off, bound, "f32", None, "dx elsewhere")
    _grad_check(None, dw, dz, ww, w64, off, bound, None, "f32", "dw elsewhere")


# few rows (split contraction), 64 x 64 to 256 x 256 tiles
@pytest.mark.parametrize("M,N,K", [(40, 72, 136), (300, 264, 136), (2048, 1024, 1033), (4096, 2048, 2048)])
def test_dense_backward(d, M, N, K):
    banner(f"dense, infinite x and w: {M} {N} {K}")
    r = np.random.default_rng(M)
    x, x64 = _mat(r, M, K)
    w, w64 = _mat(r, N, K, 0.1)
    dy, dy64 = _mat(r, M, N, 0.1)
    z, z64 = _mat(r, M, N, 1.5)
    h, h64 = _mat(r, M, N, 1.5)
    da, da64 = _mat(r, M, N // 2, 0.1)
    forms = {"linear": od.linear_backward(dy64, x64, w64, z64, "silu")[3], "gated": od.gated_linear_backward(da64, x64, w64, h64, "silu")[2]}
    x[5, 7] = float("inf")
    w[3, 11] = -float("inf")
    x64[:, 7], w64[:, 11] = 0, 0
    for form, dz in forms.items():
        if form == "linear":
            dx, dw, _ = d.linear_backward(dy, x, w, z, "silu", F32, F32)
        else:
            dx, dw = d.gated_linear_backward(da, x, w, h, "silu", F32, F32)
        _signs(dw[:, 7], dz[5], form + " dw")
        _signs(dx[:, 11], -dz[:, 3], form + " dx")
        dx[:, 11], dw[:, 7] = 0, 0
        _dense_check(dx, dw, None, (dz @ w64, dz.T @ x64, None, dz), None, x64, w64, True, "f32", "f32", form)
