"""GPU parity of the routed experts' products outside FP8 against the float64
oracle.

Bounds, with the unit roundoffs u = 2^-24 (float32) and v = 2^-8 (bf16), as for
the dense operators: 16 u |a| |b| for a product of bf16 values summed in
float32; 4 v sqrt(sum a_k^2 b_k^2) where an operand (dh) is rounded to bf16 on the
way; 2^-20 of the value for activations; u or v of the value for an output.
Integer products are exact: their sum is rounded to float32 once, and multiplied
by two scales, 3 u of the value, before the output's rounding.
"""

import numpy as np
import pytest
import torch

from gpu_util import banner, host
from oracle import dense as od
from oracle import experts as oe
from oracle import route as oroute
from test_gpu_dense import DT, U, V, _close, _mat, _norms, _vec

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "relu", "none")


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def _offsets(sizes):
    o = np.concatenate([[0], np.cumsum(sizes)])
    return o, _i32(o)


def _experts(r, G, N, K, std=0.1, pad=0, offset=0):
    w, _ = _mat(r, G * N, K, std, "bf16", pad, offset)
    w = w.unflatten(0, (G, N))
    return w, host(w).astype(np.float64)


def _per_row(off, R, f, *shape):
    """Bounds row by row: f(group, slice) over the groups' rows."""
    out = np.full((R,) + shape, np.nan)
    for g, b, e in oe.spans(off, R):
        if e > b:
            out[b:e] = f(g, slice(b, e))
    return out


def _linear_bound(x64, w64, off):
    return _per_row(off, x64.shape[0], lambda g, p: 16 * U * _norms(x64[p], w64[g]), w64.shape[1])


def _check_rows(got, want, bound, off, dtype, what):
    """The rows of the groups; those behind the last as they were (NaN)."""
    end = want.shape[0] if off is None else int(off[-1])
    _close(got[:end], want[:end], bound[:end], dtype, what)
    assert torch.isnan(got[end:]).all(), what + ": rows behind the last group"


def _nan(R, N, dtype="bf16", pad=0):
    return torch.full((R, N + pad), float("nan"), dtype=DT[dtype], device="cuda")[:, :N]


# sizes of the groups, rows behind the last one, source rows (0: no index)
GROUPS = [
    ([1], 0, 0), ([5], 2, 3), ([0, 0, 1], 0, 4), ([3, 0, 64, 65, 0, 1], 5, 40), ([63, 1, 129, 0], 0, 0),
    ([0] * 20 + [7] + [0] * 300 + [2, 0, 1] + [0] * 40, 1, 6), ([1] * 130, 0, 9), ([257, 30, 513], 3, 200),
    ([2] * 1024, 0, 50),
]


def _sources(r, R, n):
    """(source rows, index or None, index on the device): rows repeat, and some
    indices are outside the source."""
    if n == 0:
        return R, None, None
    rows = r.integers(0, n, R)
    if R > 3:
        rows[1], rows[2] = n, -1
    return n, rows, _i32(rows)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 3), (64, 64), (130, 72), (257, 515), (72, 1000)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS, ids=range(len(GROUPS)))
def test_grouped_linear(d, sizes, extra, n, N, K):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R * 3 + N + K)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, n)
    x, x64 = _mat(r, n, K)
    w, w64 = _experts(r, G, N, K)
    want = oe.grouped_linear(x64, w64, off, rows)
    bound = _linear_bound(oe.take(x64, rows), w64, off)
    for out in ("bf16", "f32"):
        banner(f"grouped_linear groups {G} rows {R} of {n}, {N}x{K} {out}")
        y = d.grouped_linear(x, w, doff, drows, y=_nan(R, N, out))
        _check_rows(y, want, bound, off, out, out)
        assert torch.equal(d.grouped_linear(x, w, doff, drows, DT[out])[:off[-1]], y[:off[-1]]), "equal bits"


def _gated_check(a, h, x64, w64, scale64, off, kind, out, what):
    wa, wh = oe.grouped_gated_linear(x64, w64, off, kind, None, scale64)
    I = wa.shape[1]
    hb = _linear_bound(x64, w64, off)
    if h is not None:
        _close(h[:off[-1]], wh[:off[-1]], hb[:off[-1]], "bf16", what + " h")
    g, u = wh[:, :I], wh[:, I:]
    f = np.abs(od.act(kind, g))
    s = 1.0 if scale64 is None else np.abs(scale64)[:, None]
    ab = s * (1.13 * hb[:, :I] * (np.abs(u) + hb[:, I:]) + f * hb[:, I:] + (2.0 ** -20 + 2 * U) * f * np.abs(u))
    _check_rows(a, wa, ab, off, out, what + " a")


@pytest.mark.parametrize("I,H", [(1, 1), (5, 9), (32, 64), (70, 136), (343, 1001), (129, 515)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS[:8], ids=range(8))
def test_grouped_gated_linear(d, sizes, extra, n, I, H):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R * 3 + I + H)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, n)
    x, x64 = _mat(r, n, H)
    w, w64 = _experts(r, G, 2 * I, H)
    s, s64 = _vec(r, R, 0.3, 1.0)
    x64 = oe.take(x64, rows)
    for i, out in enumerate(("bf16", "f32")):
        kind = ACTS[(R + I + i) % 4]
        banner(f"grouped_gated_linear groups {G} rows {R} of {n}, {I}x{H} {kind} {out}")
        a, h = d.grouped_gated_linear(x, w, doff, kind, drows, s, a=_nan(R, I, out), save_h=True)
        _gated_check(a, h, x64, w64, s64, off, kind, out, f"{kind} {out}")
        a2, none = d.grouped_gated_linear(x, w, doff, kind, drows, s, DT[out])
        assert none is None and torch.equal(a2[:off[-1]], a[:off[-1]])
    a, _ = d.grouped_gated_linear(x, w, doff, "silu", drows, a=_nan(R, I))
    _gated_check(a, None, x64, w64, None, off, "silu", "bf16", "no scale")


def _grad_check(dx, dw, dz, x64, w64, off, rounded, dxt, dwt, what):
    """dx = dz W, dW = dz^T x by groups, from the rows dz and x in float64;
    rounded: dz's relative rounding on its way into the products (0: exact)."""
    R = x64.shape[0]
    if dx is not None:
        want = _per_row(off, R, lambda g, p: dz[p] @ w64[g], x64.shape[1])
        b = _per_row(off, R, lambda g, p: 16 * U * _norms(dz[p], w64[g].T) +
                     rounded * np.sqrt((dz[p] ** 2) @ (w64[g] ** 2)), x64.shape[1])
        _check_rows(dx, want, b, off, dxt, what + " dx")
    if dw is not None:
        for g, b, e in oe.spans(off, R):
            p, q = dz[b:e], x64[b:e]
            bound = 16 * U * _norms(p.T, q.T) + rounded * np.sqrt((p.T ** 2) @ (q ** 2))
            _close(dw[g], p.T @ q, bound, dwt, f"{what} dw[{g}]")


@pytest.mark.parametrize("N,K", [(1, 1), (9, 5), (64, 72), (130, 257), (515, 136)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS[:8], ids=range(8))
def test_grouped_linear_backward(d, sizes, extra, n, N, K):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R + 5 * N + K)
    off, doff = _offsets(sizes)
    n_dy, rows, drows = _sources(r, R, n)
    dy, dy64 = _mat(r, n_dy, N, 0.1)
    w, w64 = _experts(r, G, N, K)
    x, x64 = _mat(r, R, K)
    dz = oe.take(dy64, rows)
    for dxt, dwt in (("bf16", "f32"), ("f32", "bf16")):
        banner(f"grouped_linear_backward groups {G} rows {R} of {n_dy}, {N}x{K} {dxt} {dwt}")
        dx, dw = d.grouped_linear_backward(dy, x, w, doff, dy_rows=drows, dx=_nan(R, K, dxt), dw_dtype=DT[dwt])
        _grad_check(dx, dw, dz, x64, w64, off, 0.0, dxt, dwt, dxt)
    # x by index too, one gradient at a time
    nx, xrows, dxrows = _sources(r, R, max(1, R // 2))
    x, x64 = _mat(r, nx, K)
    dx, none = d.grouped_linear_backward(dy, x, w, doff, dxrows, drows, dx=_nan(R, K), need_dw=False)
    assert none is None
    none, dw = d.grouped_linear_backward(dy, x, w, doff, dxrows, drows, need_dx=False)
    assert none is None
    _grad_check(dx, dw, dz, oe.take(x64, xrows), w64, off, 0.0, "bf16", "f32", "both by index")
    assert torch.equal(dw, d.grouped_linear_backward(dy, x, w, doff, dxrows, drows, need_dx=False)[1]), "equal bits"


@pytest.mark.parametrize("I,H", [(1, 1), (5, 9), (36, 64), (343, 257), (128, 136)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS[:8], ids=range(8))
def test_grouped_gated_linear_backward(d, sizes, extra, n, I, H):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R + 5 * I + H)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, n)
    x, x64 = _mat(r, n, H)
    w, w64 = _experts(r, G, 2 * I, H)
    h, h64 = _mat(r, R, 2 * I, 1.5)
    da, da64 = _mat(r, R, I, 0.1)
    s, s64 = _vec(r, R, 0.3, 1.0)
    x64 = oe.take(x64, rows)
    end = off[-1]
    f32, b16 = torch.float32, torch.bfloat16
    one, two = 4 * V + 2.0 ** -19, 4 * V * V + 2.0 ** -19
    for i, (dxt, dwt, dz_dtype, rounded) in enumerate((("bf16", "bf16", None, one), ("f32", "f32", None, two),
                                                       ("f32", "f32", b16, one))):
        kind = ACTS[(R + I + i) % 4]
        banner(f"grouped_gated_linear_backward groups {G} rows {R} of {n}, {I}x{H} {kind} {dxt} {dz_dtype}")
        dx, dw, ds = d.grouped_gated_linear_backward(da, x, w, h, doff, kind, drows, s, dx=_nan(R, H, dxt),
                                                     dw_dtype=DT[dwt], need_dscale=True, dz_dtype=dz_dtype)
        _, _, wds, dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off, kind, None, s64)
        _grad_check(dx, dw, dz, x64, w64, off, rounded, dxt, dwt, f"{kind} {dxt}")
        terms = np.abs(da64 * od.act(kind, h64[:, :I]) * h64[:, I:]).sum(1)
        _close(ds[:end], wds[:end], ((2.0 ** -20 + (I / 256 + 30) * U) * terms)[:end], "f32", "dscale")
        again = d.grouped_gated_linear_backward(da, x, w, h, doff, kind, drows, s, DT[dxt], DT[dwt], need_dscale=True,
                                                dz_dtype=dz_dtype)
        assert torch.equal(again[0][:end], dx[:end]) and torch.equal(again[1], dw) and torch.equal(again[2][:end], ds[:end])
    # alone: the scales' gradient; no scale
    _, _, ds2 = d.grouped_gated_linear_backward(da, x, w, h, doff, kind, drows, s, need_dx=False, need_dw=False,
                                                need_dscale=True)
    assert torch.equal(ds2[:end], ds[:end])
    dx, dw, none = d.grouped_gated_linear_backward(da, x, w, h, doff, "silu", drows, dx=_nan(R, H), dw_dtype=b16)
    assert none is None
    dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off, "silu")[3]
    _grad_check(dx, dw, dz, x64, w64, off, one, "bf16", "bf16", "no scale")


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 4), (3, 0), (1, 1)])
@pytest.mark.parametrize("indexed", [False, True])
def test_strides(d, pad, offset, indexed):
    """Rows of wider buffers whose padding is NaN, pointers of every alignment."""
    sizes, N, K = [70, 0, 33, 100], 264, 136
    banner(f"grouped strides {pad} {offset} {indexed}")
    R, G = sum(sizes), len(sizes)
    r = np.random.default_rng(7)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, 50 if indexed else 0)
    x, x64 = _mat(r, n, K, 1.0, "bf16", pad, offset)
    w, w64 = _experts(r, G, N, K, 0.1, pad, offset)
    dy, dy64 = _mat(r, R, N, 0.1, "bf16", pad, offset)
    y, _ = _mat(r, R, N, 1.0, "bf16", pad, offset)
    xr = oe.take(x64, rows)
    d.grouped_linear(x, w, doff, drows, y=y)
    _check_rows(y, oe.grouped_linear(xr, w64, off), _linear_bound(xr, w64, off), off, "bf16", "y")
    assert torch.isnan(y.as_strided((R - 1, pad), y.stride(), y.storage_offset() + N)).all()
    dx, _ = _mat(r, R, K, 1.0, "f32", pad, offset)
    dw, _ = _experts(r, G, N, K, 0.1, pad, offset)
    d.grouped_linear_backward(dy, x, w, doff, drows, dx=dx, dw=dw)
    _grad_check(dx, dw, dy64, xr, w64, off, 0.0, "f32", "bf16", "strided")
    assert torch.isnan(dx.as_strided((R - 1, pad), dx.stride(), dx.storage_offset() + K)).all()
    assert torch.isnan(dw.as_strided((G * N - 1, pad), (dw.stride(1), 1), dw.storage_offset() + K)).all()
    s, s64 = _vec(r, R + 1, 0.3, 1.0)
    a, _ = _mat(r, R, N // 2, 1.0, "f32", pad, offset)
    a, h = d.grouped_gated_linear(x, w, doff, "silu", drows, s[1:], a=a, save_h=True)
    _gated_check(a, h, xr, w64, s64[1:], off, "silu", "f32", "gated")
    h, h64 = _mat(r, R, N, 1.5, "bf16", pad, offset)
    da, da64 = _mat(r, R, N // 2, 0.1, "bf16", pad, offset)
    got = d.grouped_gated_linear_backward(da, x, w, h, doff, "gelu", drows, s[1:], dx=dx, dw13=dw)
    dz = oe.grouped_gated_linear_backward(da64, xr, w64, h64, off, "gelu", None, s64[1:])[3]
    _grad_check(got[0], got[1], dz, xr, w64, off, 4 * V + 2.0 ** -19, "f32", "bf16", "gated strided")


def test_one_expert_without_offsets(d):
    banner("grouped, one expert without offsets")
    r = np.random.default_rng(1)
    x, x64 = _mat(r, 77, 72)
    w, w64 = _experts(r, 1, 130, 72)
    dy, dy64 = _mat(r, 77, 130, 0.1)
    y = d.grouped_linear(x, w, None)
    _check_rows(y, x64 @ w64[0].T, _linear_bound(x64, w64, None), None, "bf16", "y")
    assert torch.equal(y, d.grouped_linear(x, w[0], None))
    dx, dw = d.grouped_linear_backward(dy, x, w, None)
    _grad_check(dx, dw, dy64, x64, w64, None, 0.0, "bf16", "f32", "one expert")
    with pytest.raises(ValueError):
        d.grouped_linear(x, w.expand(2, 130, 72).contiguous(), None)


def test_rows_outside_the_first_and_last_group(d):
    """Groups that begin after row 0: the rows before them belong to none."""
    banner("grouped, rows before the first group")
    r = np.random.default_rng(2)
    off = np.array([5, 40, 40, 90])
    R, N, K = 100, 72, 136
    x, x64 = _mat(r, R, K)
    w, w64 = _experts(r, 3, N, K)
    dy, dy64 = _mat(r, R, N, 0.1)
    x[:5] = float("nan")     # in no sum
    dy[90:] = float("nan")
    y = d.grouped_linear(x, w, _i32(off), y=_nan(R, N))
    want = oe.grouped_linear(x64, w64, off)
    _close(y[5:90], want[5:90], _linear_bound(x64, w64, off)[5:90], "bf16", "y")
    assert torch.isnan(y[:5]).all() and torch.isnan(y[90:]).all()
    dx, dw = d.grouped_linear_backward(dy, x, w, _i32(off), dx=_nan(R, K))
    assert torch.isnan(dx[:5]).all() and torch.isnan(dx[90:]).all()
    for g, b, e in oe.spans(off, R):
        _close(dw[g], dy64[b:e].T @ x64[b:e], 16 * U * _norms(dy64[b:e].T, x64[b:e].T), "f32", f"dw[{g}]")
    h, h64 = _mat(r, R, N, 1.5)
    da, da64 = _mat(r, R, N // 2, 0.1)
    da[:5], h[90:] = float("nan"), float("nan")
    dx, dw, _ = d.grouped_gated_linear_backward(da, x, w, h, _i32(off), dw_dtype=torch.bfloat16)
    dz = oe.grouped_gated_linear_backward(da64, x64, w64, h64, off)[3]
    for g, b, e in oe.spans(off, R):
        p, q = dz[b:e], x64[b:e]
        _close(dw[g], p.T @ q, 16 * U * _norms(p.T, q.T) + (4 * V + 2.0 ** -19) * np.sqrt((p.T ** 2) @ (q ** 2)), "bf16",
               f"gated dw[{g}]")


def test_offsets_that_break_the_rule_stay_inside_the_buffers(d):
    """Unspecified results, but no access outside: the rows around an output in
    its buffer stay as they were."""
    banner("grouped, offsets out of range and falling")
    r = np.random.default_rng(3)
    R, N, K = 90, 72, 64
    x, _ = _mat(r, R, K)
    w, _ = _experts(r, 3, N, K)
    dy, _ = _mat(r, R, N)
    for off in ([-7, 30, 20, 500], [90, 60, 30, 0], [0, 2 ** 31 - 1, -2 ** 31, 90]):
        buf = _nan(R + 20, N)
        d.grouped_linear(x, w, _i32(off), y=buf[10:10 + R])
        bufx = _nan(R + 20, K)
        _, dw = d.grouped_linear_backward(dy, x, w, _i32(off), dx=bufx[10:10 + R])
        h = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
        _, dw13, _ = d.grouped_gated_linear_backward(dy[:, :N // 2], x, w, h, _i32(off), need_dscale=True)
        torch.cuda.synchronize()
        for b in (buf, bufx):
            assert torch.isnan(b[:10]).all() and torch.isnan(b[10 + R:]).all()
        assert torch.isfinite(dw).all() and torch.isfinite(dw13).all()


def test_nan_and_infinity_stay_in_their_rows(d):
    banner("grouped, NaN rows")
    r = np.random.default_rng(4)
    off, doff = _offsets([40, 50])
    x, _ = _mat(r, 90, 136)
    w, _ = _experts(r, 2, 72, 136)
    x[7, 3] = float("nan")
    x[60, 9] = float("inf")
    y = d.grouped_linear(x, w, doff)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 60] and torch.isnan(y[7]).all()
    _, dw = d.grouped_linear_backward(y.nan_to_num(0, 1, -1), x, w, doff, need_dx=False)
    assert torch.isnan(dw[0][:, 3]).all() and torch.isfinite(dw[0][:, :3]).all() and torch.isfinite(dw[1][:, :9]).all()


def test_offsets_past_32_bits(d):
    """Weights and gathered rows past 2^32 bytes, and rows by index that span
    more than the copies' offsets reach."""
    ld, N, K, G = 4194304, 130, 136, 5
    banner("grouped, offsets past 32 bits")
    r = np.random.default_rng(5)
    big = torch.zeros((G * N * ld,), dtype=torch.bfloat16, device="cuda").view(G * N, ld)
    w = big[:, 64:64 + K].unflatten(0, (G, N))
    w.copy_(torch.from_numpy(r.standard_normal((G, N, K)).astype(np.float32) * np.float32(0.1)))
    w64 = host(w).astype(np.float64)
    x = big[:300, 4096:4096 + K]
    x.copy_(torch.from_numpy(r.standard_normal((300, K)).astype(np.float32)))
    x64 = host(x).astype(np.float64)
    sizes = [100, 0, 150, 1, 99]
    R = sum(sizes)
    off, doff = _offsets(sizes)
    rows = r.integers(0, 300, R)
    xr = oe.take(x64, rows)
    y = d.grouped_linear(x, w, doff, _i32(rows))
    _check_rows(y, oe.grouped_linear(xr, w64, off), _linear_bound(xr, w64, off), off, "bf16", "y")
    dy, dy64 = _mat(r, R, N, 0.1)
    dw = big[:, 8192:8192 + K].unflatten(0, (G, N))
    dx, dw = d.grouped_linear_backward(dy, x, w, doff, _i32(rows), dw=dw)
    _grad_check(dx, dw, dy64, xr, w64, off, 0.0, "bf16", "bf16", "past 32 bits")


def test_no_rows(d):
    banner("grouped, no rows")
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    w, off = e(3, 32, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert d.grouped_linear(e(0, 64), w, off).shape == (0, 32)
    assert d.grouped_linear(e(5, 64), w, off, none).shape == (0, 32)
    dx, dw = d.grouped_linear_backward(e(0, 32), e(0, 64), w, off)
    assert dx.shape == (0, 64) and not dw.any() and dw.shape == (3, 32, 64)
    a, h = d.grouped_gated_linear(e(0, 64), w, off, save_h=True)
    assert a.shape == (0, 16) and h.shape == (0, 32)
    dx, dw, ds = d.grouped_gated_linear_backward(e(0, 16), e(0, 64), w, h, off, need_dscale=True)
    assert dx.shape == (0, 64) and not dw.any() and ds.shape == (0,)
    # rows, but none in a group
    y = _nan(9, 32)
    d.grouped_linear(e(9, 64), w, off, y=y)
    assert torch.isnan(y).all()
    _, dw = d.grouped_linear_backward(e(9, 32), e(9, 64), w, off, dw=_nan(96, 64, "f32").unflatten(0, (3, 32)))
    assert not dw.any()
    q, s = d.quant_rows_int8(e(0, 64))
    assert d.int8_linear(q, s, torch.zeros((3, 32, 64), dtype=torch.int8, device="cuda"),
                         torch.ones((3, 32), device="cuda"), off).shape == (0, 32)


# ---------------------------------------------------------------------------
# 8-bit integers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (40, 64), (5, 65), (129, 512), (7, 513), (33, 2048), (9, 2056),
                                       (3, 4099), (17, 7168), (2, 8192), (3, 8200), (2, 40001)])
def test_quant_rows_int8(d, rows, cols, dtype):
    banner(f"quant_rows_int8 {rows}x{cols} {dtype}")
    r = np.random.default_rng(rows + cols)
    for pad, offset in ((0, 0), (3, 1)):
        x, x64 = _mat(r, rows, cols, 3.0, dtype, pad, offset)
        if rows > 2:
            x[1] = 0
            x[2, :cols // 2] = -0.0
            x64 = host(x).astype(np.float64)
        q, s = d.quant_rows_int8(x)
        wq, ws = oe.quant_int8(x64)
        assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)
        buf = torch.full((rows, cols + 5), 99, dtype=torch.int8, device="cuda")
        d.quant_rows_int8(x, buf[:, 1:1 + cols])
        assert torch.equal(buf[:, 1:1 + cols], q) and (buf[:, 0] == 99).all() and (buf[:, 1 + cols:] == 99).all()


def test_quant_rows_int8_of_extremes(d):
    """Ties, the smallest and largest floats, rows that are not finite."""
    banner("quant_rows_int8 extremes")
    tiny, big = np.float32(2.0 ** -149), np.float32(3.4e38)
    rows = [[127, -63.5, 0.5, 1.5, -2.5, 126.5], [tiny, 0, -tiny, 0, 0, 0], [190 * tiny, -190 * tiny, 64 * tiny, 0, 0, 0],
            [big, -big, big / 254, 1, 0, -0.0], [1, np.nan, 2, 3, 4, 5], [1, np.inf, 2, 3, 4, 5], [-np.inf] * 6,
            [0] * 6, [1e-38, 1e-39, 1e-40, 5e-41, 0, 0]]
    x = np.array(rows, np.float32)
    x = np.concatenate([x, np.random.default_rng(0).standard_normal((2000, 6)).astype(np.float32) *
                        2.0 ** np.random.default_rng(1).integers(-140, 120, (2000, 1))]).astype(np.float32)
    q, s = d.quant_rows_int8(torch.from_numpy(x).cuda())
    wq, ws = oe.quant_int8(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws, equal_nan=True)
    y = d.int8_linear(q[3:9], s[3:9], torch.ones((4, 6), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"))
    assert torch.isnan(y[1:4]).all() and torch.isfinite(y[4:]).all()


def _codes(r, *shape):
    q = r.integers(-127, 128, shape)
    return torch.from_numpy(q.astype(np.int8)).cuda(), q.astype(np.float64)


def _scales(r, *shape):
    s = (r.random(shape) * 0.1 + 0.01).astype(np.float32)
    return torch.from_numpy(s).cuda(), s.astype(np.float64)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 3), (64, 128), (130, 72), (257, 515), (72, 2064)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS, ids=range(len(GROUPS)))
def test_int8_linear(d, sizes, extra, n, N, K):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R * 3 + N + K)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, n)
    (x, x64), (w, w64) = _codes(r, n, K), _codes(r, G, N, K)
    (xs, xs64), (ws, ws64) = _scales(r, n), _scales(r, G, N)
    want, _ = oe.int8_linear(x64, xs64, w64, ws64, off, rows)
    for out in ("bf16", "f32"):
        banner(f"int8_linear groups {G} rows {R} of {n}, {N}x{K} {out}")
        y = d.int8_linear(x, xs, w, ws, doff, drows, y=_nan(R, N, out))
        _check_rows(y, want, 3.01 * U * np.abs(want), off, out, out)


@pytest.mark.parametrize("I,H", [(1, 1), (5, 9), (32, 128), (70, 136), (343, 1001)])
@pytest.mark.parametrize("sizes,extra,n", GROUPS[:8], ids=range(8))
def test_int8_gated_linear(d, sizes, extra, n, I, H):
    R, G = sum(sizes) + extra, len(sizes)
    r = np.random.default_rng(R * 3 + I + H)
    off, doff = _offsets(sizes)
    n, rows, drows = _sources(r, R, n)
    (x, x64), (w, w64) = _codes(r, n, H), _codes(r, G, 2 * I, H)
    (xs, xs64), (ws, ws64) = _scales(r, n), _scales(r, G, 2 * I)
    ws, ws64 = ws / H, ws64 / H
    ws64 = host(ws).astype(np.float64)
    s, s64 = _vec(r, R, 0.3, 1.0)
    h, _ = oe.int8_linear(x64, xs64, w64, ws64, off, rows)
    g, u = h[:, :I], h[:, I:]
    for i, out in enumerate(("bf16", "f32")):
        kind = ACTS[(R + I + i) % 4]
        banner(f"int8_gated_linear groups {G} rows {R} of {n}, {I}x{H} {kind} {out}")
        a = d.int8_gated_linear(x, xs, w, ws, doff, kind, drows, s, a=_nan(R, I, out))
        f = np.abs(od.act(kind, g))
        hb = 3.01 * U * np.abs(h)
        bound = np.abs(s64)[:, None] * (1.13 * hb[:, :I] * (np.abs(u) + hb[:, I:]) + f * hb[:, I:] +
                                        (2.0 ** -20 + 2 * U) * f * np.abs(u))
        _check_rows(a, s64[:, None] * od.act(kind, g) * u, bound, off, out, f"{kind} {out}")


def test_int8_strides_and_dense_form(d):
    banner("int8 strides, without offsets")
    r = np.random.default_rng(8)
    M, N, K = 203, 264, 136
    for pad, at in ((8, 0), (24, 16), (3, 0), (1, 1)):
        xb, xb64 = _codes(r, M, K + pad + at)
        wb, wb64 = _codes(r, N, K + pad + at)
        x, w, x64, w64 = xb[:, at:at + K], wb[:, at:at + K], xb64[:, at:at + K], wb64[:, at:at + K]
        (xs, xs64), (ws, ws64) = _scales(r, M), _scales(r, N)
        want = xs64[:, None] * ws64 * (x64 @ w64.T)
        y = d.int8_linear(x, xs, w, ws, out_dtype=torch.float32)
        _close(y, want, 3.01 * U * np.abs(want), "f32", f"pad {pad} at {at}")


def test_int8_sums_of_the_longest_contraction(d):
    """The largest sums that the longest K gives, exact in 32 bits."""
    banner("int8, K 131071")
    K = 131071
    x = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    x[1], w[2] = 127, 127
    x[2, 1::2] = 127
    one = lambda n: torch.ones(n, device="cuda")
    y = d.int8_linear(x, one(3), w, one(5), out_dtype=torch.float32)
    want = host(x).astype(np.float64) @ host(w).astype(np.float64).T
    assert np.abs(want).max() > 2 ** 30
    _close(y, want, np.abs(want) * U, "f32", "longest sums")
    with pytest.raises(d.DsmoeError):
        big = torch.zeros((1, K + 1), dtype=torch.int8, device="cuda")
        d.int8_linear(big, one(1), big, one(1))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,K,H", [(1, 1, 1, 8), (9, 16, 2, 64), (300, 64, 8, 64), (5, 1024, 32, 8)])
def test_router_backward(d, T, E, K, H):
    banner(f"router_backward {T} {E} {K}")
    r = np.random.default_rng(T)
    z = r.standard_normal((T, E)).astype(np.float32) * 2
    top = np.stack([r.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    dg = r.standard_normal((T, K)).astype(np.float32)
    got = d.router_backward(torch.from_numpy(dg).cuda(), _i32(top), torch.from_numpy(z).cuda())
    s = 1 / (1 + np.exp(-np.take_along_axis(z.astype(np.float64), top, 1)))
    total = s.sum(1, keepdims=True)
    bound = np.zeros((T, E))
    # dgate and the mean each rounded, K sums: of the terms' sizes
    np.put_along_axis(bound, top, (2 * K + 12) * U * (np.abs(dg) + (np.abs(dg) * s).sum(1, keepdims=True) / total) / total * s, 1)
    _close(got, oe.router_backward(dg, top, z), bound, "f32", "dlogits")


def _layer(d, r, T, H, I, E, K, n_shared, scale=0.1):
    x, x64 = _mat(r, T, H)
    w13, w13_64 = _experts(r, E + n_shared, 2 * I, H, scale)
    w2, w2_64 = _experts(r, E + n_shared, H, I, scale)
    logits = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).cuda()
    routing = d.route(logits, torch.zeros(E, device="cuda"), 1, 1, K)
    return x, x64, w13, w13_64, w2, w2_64, logits, routing


@pytest.mark.parametrize("n_shared", [0, 1])
def test_the_experts_pass_and_its_gradients(d, n_shared):
    T, H, I, E, K = 200, 136, 72, 7, 3
    banner(f"moe_ffn forward and backward, shared {n_shared}")
    r = np.random.default_rng(12)
    x, x64, w13, w13_64, w2, w2_64, logits, routing = _layer(d, r, T, H, I, E, K, n_shared, 0.15)
    y, saved = d.moe_ffn_forward(x, routing, w13, w2, n_shared=n_shared, training=True)
    y2, none = d.moe_ffn_forward(x, routing, w13, w2, n_shared=n_shared)
    assert none is None and torch.equal(y, y2)
    top, gates = host(routing["topk_idx"]), host(routing["gates"]).astype(np.float64)

    def forward(x64=x64, w13_64=w13_64, w2_64=w2_64, gates=gates):
        return oe.moe_ffn(x64, w13_64[:E], w2_64[:E], top, gates, shared=(w13_64[E], w2_64[E]) if n_shared else None)

    want = forward()
    # a and o rounded to bf16 on the way: v of each term of the sums, independent
    a64 = host(saved["a"]).astype(np.float64)
    o = oe.grouped_linear(a64, w2_64, host(saved["offsets"]))
    size = np.zeros((T, H))
    np.add.at(size, host(saved["perm"]), o * o)
    ab = np.zeros((T, H))
    np.add.at(ab, host(saved["perm"]), oe.grouped_linear(a64 * a64, w2_64 * w2_64, host(saved["offsets"])))
    _close(y, want, 4 * V * (np.sqrt(size) + np.sqrt(ab)) + 2.0 ** -16 * np.sqrt(ab), "bf16", "y")
    dy, dy64 = _mat(r, T, H, 0.1)
    got = d.moe_ffn_backward(dy, x, routing, w13, w2, saved, logits=logits)
    z64 = host(logits).astype(np.float64)

    def loss(z64=z64, **v):
        s = 1 / (1 + np.exp(-np.take_along_axis(z64, top, 1)))
        v.setdefault("gates", s / s.sum(1, keepdims=True))
        return float((forward(**v) * dy64).sum())

    # along random directions, as in the dense sub-layer's test: roundings to
    # bf16 of a, da, dh, dx per row and h, five of v per element
    for name, arr, key in (("x64", x64, "dx"), ("w13_64", w13_64, "dw13"), ("w2_64", w2_64, "dw2"), ("gates", gates, "dgates"),
                           ("z64", z64, "dlogits")):
        v = r.standard_normal(arr.shape)
        num = (loss(**{name: arr + 1e-5 * v}) - loss(**{name: arr - 1e-5 * v})) / 2e-5
        terms = host(got[key]).astype(np.float64) * v
        assert abs(terms.sum() - num) <= 8 * 5 * V * np.linalg.norm(terms), (key, terms.sum(), num)


@pytest.mark.parametrize("n_shared", [0, 1])
def test_the_experts_pass_in_8_bits(d, n_shared):
    """Step by step against the same steps of the oracle on the codes that the
    quantiser gives (which it matches bit for bit)."""
    T, H, I, E, K = 200, 136, 72, 7, 3
    banner(f"moe_ffn int8, shared {n_shared}")
    r = np.random.default_rng(13)
    x, x64, w13, w13_64, w2, w2_64, _, routing = _layer(d, r, T, H, I, E, K, n_shared)
    q13, q2 = d.quant_rows_int8(w13), d.quant_rows_int8(w2)
    y = d.moe_ffn_int8_forward(x, routing, q13, q2, n_shared=n_shared)
    off, perm, scale = (host(t) for t in d.experts._routed_rows(routing, n_shared)[:3])
    codes, cs = oe.quant_int8(x64)
    w13q, w2q = host(q13[0]).astype(np.float64), host(q2[0]).astype(np.float64)
    assert np.array_equal(w13q.reshape(-1, H), oe.quant_int8(w13_64.reshape(-1, H))[0])
    h, _ = oe.int8_linear(codes, cs, w13q, host(q13[1]), off, perm)
    a64 = scale.astype(np.float64)[:, None] * od.act("silu", h[:, :I]) * h[:, I:]
    # a rounded to bf16 (v) and to codes (half a step: max / 254), each element
    # by itself, then o to bf16
    a_err = np.sqrt((V * np.abs(a64)) ** 2 + (np.abs(a64).max(1, keepdims=True) / 254) ** 2)
    w2d = w2q * host(q2[1]).astype(np.float64)[..., None]
    o = oe.grouped_linear(a64, w2d, off)
    var = oe.grouped_linear(a_err ** 2, w2d ** 2, off) + (V * o) ** 2
    want, ab = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want, perm, o)
    np.add.at(ab, perm, var)
    _close(y, want, 4 * np.sqrt(ab) + 2.0 ** -16 * np.abs(want), "bf16", "y")


def test_calls_on_other_streams_and_in_graphs(d):
    """The whole pass on a side stream, and captured with its workspaces and
    replayed with other inputs, eager work in between."""
    T, H, I, E, K = 64, 136, 70, 6, 2     # I not a multiple of 8: operands are copied first
    banner("moe_ffn on a side stream and in a graph")
    r = np.random.default_rng(14)
    x, _, w13, _, w2, _, logits, routing = _layer(d, r, T, H, I, E, K, 0)
    q13, q2 = d.quant_rows_int8(w13), d.quant_rows_int8(w2)
    dy, _ = _mat(r, T, H, 0.1)
    off, perm, scale, _ = d.experts._routed_rows(routing, 0)

    def step():
        a, h = d.grouped_gated_linear(x, w13, off, rows=perm, row_scale=scale, save_h=True)
        y = d.combine_rows(d.grouped_linear(a, w2, off), routing["inv"])
        da, dw2 = d.grouped_linear_backward(dy, a, w2, off, dy_rows=perm)
        dx, dw13, ds = d.grouped_gated_linear_backward(da, x, w13, h, off, rows=perm, row_scale=scale, need_dscale=True)
        q, s = d.quant_rows_int8(x)
        b = d.int8_gated_linear(q, s, *q13, off, rows=perm, row_scale=scale)
        return y, da, dw2, d.combine_rows(dx, routing["inv"]), dw13, ds, b, d.int8_linear(*d.quant_rows_int8(b), *q2, off)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_a_caller_s_workspace(d):
    """Operands that are copied, in the caller's workspace; too small a one is
    refused."""
    banner("grouped, the caller's workspace")
    r = np.random.default_rng(15)
    off, doff = _offsets([30, 41])
    x, _ = _mat(r, 71, 131)
    w, _ = _experts(r, 2, 67, 131)
    need = d.lib.dsmoe_grouped_linear_workspace_bytes(x.data_ptr(), 131, 71, None, w.data_ptr(), 131, 2, 71, 67, 131)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(d.grouped_linear(x, w, doff, workspace=ws), d.grouped_linear(x, w, doff))
    with pytest.raises(d.DsmoeError):
        d.grouped_linear(x, w, doff, workspace=ws[:need - 256])
    with pytest.raises(ValueError):
        d.grouped_linear(x, w, doff, workspace=torch.empty(need, device="cuda"))
