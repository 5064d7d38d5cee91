"""Every kernel of the dense products in every form (tile shape, direction,
splits of K, the cut into two launches), whole results against float64 products
on the GPU.  Bounds as derived in test_gpu_dense.py."""

import pytest
import torch

import dense_kernels as dk
from gpu_util import banner

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _close(got, want, bound, rel, what):
    lim = bound + 1.01 * rel * (want.abs() + bound)
    err = (got.double() - want).abs()
    bad = ~(err <= lim)
    print(f"[parity] {what}: worst error / bound {float((err / lim).max()):.3f}", flush=True)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def _norms(a, b):
    return a.norm(dim=1)[:, None] * b.norm(dim=1)[None, :]


@pytest.mark.parametrize("size", dk.SIZES, ids=lambda s: "-".join(map(str, s)))
def test_every_kernel(d, size):
    product, M, N, K = size
    want_kernels = dk.SIZES[size]
    assert dk.kernels(d.lib, *size) == want_kernels
    banner(f"{product} {M}x{N}x{K}: {want_kernels}")
    g = torch.Generator(device="cuda").manual_seed(M + N + K)

    def randn(rows, cols, std=1.0):
        return (torch.randn((rows, cols), generator=g, device="cuda") * std).bfloat16()

    x = randn(M, K)
    x64 = x.double()
    if product == "gated":
        w = randn(2 * N, K, 0.1)
        w64 = w.double()
        a, h = d.gated_linear(x, w, "silu", torch.float32, save_h=True)
        want, hb = x64 @ w64.t(), 16 * U * _norms(x64, w64)
        _close(h, want, hb, V, "h")
        gate, up, gb, ub = want[:, :N], want[:, N:], hb[:, :N], hb[:, N:]
        f = gate * torch.sigmoid(gate)
        bound = 1.13 * gb * (up.abs() + ub) + f.abs() * ub + 2.0 ** -20 * (f * up).abs()
        _close(a, f * up, bound, U, "a")
        again = d.gated_linear(x, w, "silu", torch.float32)[0]
        assert torch.equal(a, again)
        return
    w = randn(N, K, 0.1)
    w64 = w.double()
    if product == "y":
        bias = torch.randn((N,), generator=g, device="cuda")
        res = randn(M, N)
        z64, zb = x64 @ w64.t() + bias.double(), 16 * U * _norms(x64, w64)
        zb = zb + 2 * U * z64.abs()
        y, z = d.linear(x, w, bias, "silu", res.float(), torch.float32, save_z=True)
        _close(z, z64, zb, U, "z")
        f = z64 * torch.sigmoid(z64)
        want = f + res.double()
        _close(y, want, 1.13 * zb + 2.0 ** -20 * f.abs() + U * want.abs(), U, "y silu f32")
        want = z64 + res.double()
        for out, rel in ((torch.bfloat16, V), (torch.float32, U)):
            y, _ = d.linear(x, w, bias, residual=res.to(out), out_dtype=out)
            _close(y, want, zb + U * want.abs(), rel, f"y {out}")
            assert torch.equal(y, d.linear(x, w, bias, residual=res.to(out), out_dtype=out)[0])
        return
    dy = randn(M, N, 0.1)
    dy64 = dy.double()
    for out, rel in ((torch.bfloat16, V), (torch.float32, U)):
        dx, dw, _ = d.linear_backward(dy, x, w, dx_dtype=out, dw_dtype=out, need_dx=product == "dx",
                                      need_dw=product == "dw")
        if product == "dx":
            _close(dx, dy64 @ w64, 16 * U * _norms(dy64, w64.t()), rel, f"dx {out}")
        else:
            _close(dw, dy64.t() @ x64, 16 * U * _norms(dy64.t(), x64.t()), rel, f"dw {out}")
    again = d.linear_backward(dy, x, w, dx_dtype=out, dw_dtype=out, need_dx=product == "dx", need_dw=product == "dw")
    assert torch.equal(again[0] if product == "dx" else again[1], dx if product == "dx" else dw)
