"""Every kernel of the grouped products in every form (grouped_kernels.SIZES)
against float64: the whole result, groups of uneven sizes and without rows, rows
behind the last group, rows by index and in place."""

import numpy as np
import pytest
import torch

import grouped_kernels as gk
from gpu_util import banner, host
from oracle import experts as oe
from test_gpu_dense import DT, U, V, _mat, _vec
from test_gpu_experts import (_check_rows, _codes, _experts, _gated_check, _grad_check, _i32, _linear_bound, _nan, _offsets,
                              _scales)
from oracle import dense as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


@pytest.mark.parametrize("size", gk.SIZES, ids=lambda s: "-".join(map(str, s)).replace(" ", "_"))
def test_grouped_kernel(d, size):
    product, G, R, N, K = size
    assert gk.shape(d.lib, *size) == gk.SIZES[size]
    sizes = gk.group_sizes(G, R)
    behind = min(sizes[-1], 3)        # the last rows belong to no group
    sizes[-1] -= behind
    off, doff = _offsets(sizes)
    r = np.random.default_rng(G + N)
    n = max(1, R // 3)
    rows = r.integers(0, n, R)
    drows = _i32(rows)
    banner(f"{product} {G} groups {R} rows {N}x{K}: {gk.SIZES[size]}")
    if product in ("y", "gated"):
        w, w64 = _experts(r, G, N * (2 if product == "gated" else 1), K)
        x, x64 = _mat(r, n, K)
        xr = oe.take(x64, rows)
        # by index, then the same rows in place
        if product == "y":
            bound, want = _linear_bound(xr, w64, off), oe.grouped_linear(xr, w64, off)
            for out in ("bf16", "f32"):
                y = d.grouped_linear(x, w, doff, drows, y=_nan(R, N, out))
                _check_rows(y, want, bound, off, out, out)
                y2 = d.grouped_linear(x[drows.long()].contiguous(), w, doff, y=_nan(R, N, out, pad=5))
                assert torch.equal(y2[:off[-1]], y[:off[-1]]) and torch.isnan(y2[off[-1]:]).all()
        else:
            s, s64 = _vec(r, R, 0.3, 1.0)
            for out in ("bf16", "f32"):
                a, h = d.grouped_gated_linear(x, w, doff, "silu", drows, s, a=_nan(R, N, out), save_h=True)
                _gated_check(a, h, xr, w64, s64, off, "silu", out, out)
                a2, h2 = d.grouped_gated_linear(x[drows.long()].contiguous(), w, doff, "silu", None, s, a=_nan(R, N, out, pad=5))
                assert h2 is None and torch.equal(a2[:off[-1]], a[:off[-1]]) and torch.isnan(a2[off[-1]:]).all()
        return
    if product in ("dx", "dw"):
        w, w64 = _experts(r, G, N, K)
        dy, dy64 = _mat(r, n, N, 0.1)
        x, x64 = _mat(r, R, K)
        dz = oe.take(dy64, rows)
        kw = dict(need_dw=False) if product == "dx" else dict(need_dx=False)
        for t in ("bf16", "f32"):
            out = dict(dx=_nan(R, K, t, pad=5)) if product == "dx" else dict(dw=_nan(G * N, K, t, pad=5).unflatten(0, (G, N)))
            dx, dw = d.grouped_linear_backward(dy, x, w, doff, dy_rows=drows, **kw, **out)
            _grad_check(dx, dw, dz, x64, w64, off, 0.0, t, t, t)
        if product == "dw":
            # two products, the second added to the first: the gradient of the gated
            # form in float32
            if N % 2 == 0:
                h, h64 = _mat(r, R, N, 1.5)
                da, da64 = _mat(r, R, N // 2, 0.1)
                _, dw, _ = d.grouped_gated_linear_backward(da, x, w, h, doff, need_dx=False, dw_dtype=torch.float32)
                dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off)[3]
                _grad_check(None, dw, dz, x64, w64, off, 4 * V * V + 2.0 ** -19, None, "f32", "added")
        return
    (x, x64), (w, w64) = _codes(r, n, K), _codes(r, G, N * (2 if "gated" in product else 1), K)
    (xs, xs64), (ws, _) = _scales(r, n), _scales(r, G, w.shape[1])
    ws = ws / K
    want, _ = oe.int8_linear(x64, xs64, w64, host(ws).astype(np.float64), off, rows)
    for out in ("bf16", "f32"):
        if "gated" in product:
            s, s64 = _vec(r, R, 0.3, 1.0)
            g, u = want[:, :N], want[:, N:]
            f, hb = np.abs(od.act("silu", g)), 3.01 * U * np.abs(want)
            bound = np.abs(s64)[:, None] * (1.13 * hb[:, :N] * (np.abs(u) + hb[:, N:]) + f * hb[:, N:] +
                                            (2.0 ** -20 + 2 * U) * f * np.abs(u))
            a = d.int8_gated_linear(x, xs, w, ws, doff, "silu", drows, s, a=_nan(R, N, out, pad=5))
            _check_rows(a, s64[:, None] * od.act("silu", g) * u, bound, off, out, out)
        else:
            y = d.int8_linear(x, xs, w, ws, doff, drows, y=_nan(R, N, out, pad=5))
            _check_rows(y, want, 3.01 * U * np.abs(want), off, out, out)


# of SIZES, one of each product in 256 x 256 tiles and one in small ones
BROKEN = [("y", 130, 39000, 136, 72), ("y", 3, 65, 1000, 520), ("dx", 40, 12000, 520, 520), ("dw", 700, 14000, 264, 300),
          ("dw", 7, 5000, 520, 391), ("gated", 40, 5200, 520, 201), ("int8", 130, 39000, 136, 200)]


@pytest.mark.parametrize("size", BROKEN, ids=lambda s: "-".join(map(str, s)))
def test_offsets_that_break_the_rule(d, size):
    """Offsets that fall, that are negative or that pass R: nothing outside the result
    is written (bands of NaN on both sides), and the next call is right."""
    product, G, R, N, K = size
    r = np.random.default_rng(R)
    banner(f"{product} {G} groups {R} rows {N}x{K}: offsets that break the rule")
    bad = r.integers(-R, 2 * R, G + 1)
    bad[r.integers(0, G + 1, G // 3 + 1)] = R
    cases = [bad, bad[::-1].copy(), np.full(G + 1, -2 ** 31), np.full(G + 1, 2 ** 31 - 1),
             np.where(np.arange(G + 1) % 2, R, 0)]
    good = gk.group_sizes(G, R)
    cols = {"y": N, "dx": K, "dw": K, "gated": N, "int8": N}[product]
    rows = G * N if product == "dw" else R
    guard = 300
    buf = _nan(rows + 2 * guard, cols)
    out = buf[guard:guard + rows]
    if product == "int8":
        x, w = _codes(r, R, K)[0], _codes(r, G, N, K)[0]
        (xs, _), (ws, _) = _scales(r, R), _scales(r, G, N)
        run = lambda off: d.int8_linear(x, xs, w, ws, off, y=out)
    elif product == "dw":
        dy, x, w = _mat(r, R, N)[0], _mat(r, R, K)[0], _experts(r, G, N, K)[0]
        run = lambda off: d.grouped_linear_backward(dy, x, w, off, need_dx=False, dw=out.unflatten(0, (G, N)))
    elif product == "dx":
        dy, x, w = _mat(r, R, N)[0], _mat(r, R, K)[0], _experts(r, G, N, K)[0]
        run = lambda off: d.grouped_linear_backward(dy, x, w, off, need_dw=False, dx=out)
    else:
        x, w = _mat(r, R, K)[0], _experts(r, G, N * (2 if product == "gated" else 1), K)[0]
        run = (lambda off: d.grouped_linear(x, w, off, y=out)) if product == "y" else \
            (lambda off: d.grouped_gated_linear(x, w, off, a=out))
    run(_offsets(good)[1])
    want = out.clone()
    for c in cases:
        run(_i32(c))
        torch.cuda.synchronize()
        assert torch.isnan(buf[:guard]).all() and torch.isnan(buf[guard + rows:]).all()
    run(_offsets(good)[1])
    assert torch.equal(out, want)


def test_blocks_that_stay_in_graphs_and_on_two_streams(d):
    """y, dW and the 8-bit y in 256 x 256 tiles, several tiles a block: captured
    together and replayed with other inputs and other offsets, eager work in
    between; and on two streams at once."""
    G, R, N, K = 40, 12000, 520, 520
    assert all(gk.shape(d.lib, p, G, R, N, K) == "256x256" for p in ("y", "dw"))
    G8, R8, N8, K8 = 130, 39000, 136, 200
    assert gk.shape(d.lib, "int8", G8, R8, N8, K8) == "256x256"
    banner("grouped 256x256 in graphs and on two streams")
    r = np.random.default_rng(5)
    sets = []
    for i in range(2):
        sizes = gk.group_sizes(G, R)
        r.shuffle(sizes)
        sets.append([_mat(r, R, K)[0], _mat(r, R, N, 0.1)[0], _experts(r, G, N, K)[0], _offsets(sizes)[1],
                     _codes(r, R8, K8)[0], _scales(r, R8)[0], _codes(r, G8, N8, K8)[0], _scales(r, G8, N8)[0],
                     _offsets(gk.group_sizes(G8, R8))[1]])

    def step(x, dy, w, off, q, qs, w8, w8s, off8):
        y = d.grouped_linear(x, w, off)
        dw = d.grouped_linear_backward(dy, x, w, off, need_dx=False)[1]
        return y, dw, d.int8_linear(q, qs, w8, w8s, off8)

    want = [step(*s) for s in sets]
    held = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held)
    for i in (0, 1, 0):
        for t, s in zip(held, sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
        assert all(torch.equal(a, b) for a, b in zip(step(*sets[1 - i]), want[1 - i]))
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(*sets[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
