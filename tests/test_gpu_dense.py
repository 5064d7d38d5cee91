"""GPU parity of the dense feed-forward operators against the float64 oracle.

Bounds, with the unit roundoffs u = 2^-24 (float32: 24 significant bits) and
v = 2^-8 (bf16: 8 significant bits):

* a product c = sum_k a_k b_k of bf16 values: the products are exact in
  float32; each of the K additions rounds by at most u of a partial sum, and
  partial sums of terms of mixed sign stay near |a| |b| / sqrt(K) times a few,
  their roundings adding up as a random walk: 16 u |a| |b| (2-norms) covers
  both with room.  A dropped or doubled term is about |a| |b| / K, far above.
* an operand rounded to bf16 on the way (dz, dh): each term moves by at most
  v of itself, independently: 4 v sqrt(sum_k a_k^2 b_k^2), seven standard
  deviations of uniform roundings.
* activations and their derivatives: a few float32 ulps of their value and of
  their argument's effect (|f'| <= 1.13): 2^-20 of the value.
* layer norm: sums of one row in float32, depth at most 64: 64 u of the sums'
  absolute terms.
* an output rounded to its type: u or v of the value.
"""

import math

import numpy as np
import pytest
import torch

from gpu_util import banner, host
from oracle import dense as od

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT_REL = {"bf16": V * 1.01, "f32": U * 1.01}


@pytest.fixture(scope="module")
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def _mat(r, rows, cols, std=1.0, dtype="bf16", pad=0, offset=0, fill=float("nan")):
    """(device view [rows][cols] whose row padding holds `fill`, float64 values)."""
    buf = torch.full((offset + max(rows, 1) * (cols + pad),), fill, dtype=DT[dtype], device="cuda")
    v = buf[offset:].view(max(rows, 1), cols + pad)[:rows, :cols]
    v.copy_(torch.from_numpy(r.standard_normal((rows, cols)).astype(np.float32) * np.float32(std)))
    return v, host(v).astype(np.float64)


def _vec(r, n, std=1.0, mean=0.0, dtype="f32"):
    t = torch.from_numpy((r.standard_normal(n) * std + mean).astype(np.float32)).to(DT[dtype]).cuda()
    return t, host(t).astype(np.float64)


def _close(got, want, bound, dtype, what):
    got = host(got).astype(np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = np.abs(got - want)
    lim = bound + OUT_REL[dtype] * (np.abs(want) + bound)
    bad = ~(err <= lim)
    if got.size:
        with np.errstate(divide="ignore", invalid="ignore"):
            print(f"[parity] {what}: worst error / bound {float(np.nanmax(np.where(lim > 0, err / lim, 0))):.3f}", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first {np.argwhere(bad)[0]}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}"


def _norms(a, b):
    """|a_m| |b_n| of the rows of a and b."""
    return np.linalg.norm(a, axis=1)[:, None] * np.linalg.norm(b, axis=1)[None, :]


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

NORM_SHAPES = [  # rows, cols: each register layout, its edges, the long rows
    (1, 1), (1, 7168), (3, 7), (5, 64), (64, 512), (65, 513), (7, 1000), (130, 1024), (4, 1025), (9, 2048), (5, 2056),
    (33, 4096), (6, 4104), (17, 7168), (2, 8192), (3, 8200), (2, 16384), (2, 16392), (2, 32768), (2, 32776), (3, 40001),
    (1037, 1001), (3000, 136)]


def _norm_inputs(seed, rows, cols, dtype, pad, offset=0):
    r = np.random.default_rng(seed)
    x, x64 = _mat(r, rows, cols, 1.0, dtype, pad, offset)
    big = np.arange(cols) % 37 == 5           # a few large channels, a mean off 0
    x.mul_(torch.from_numpy(np.where(big, 30.0, 1.0).astype(np.float32)).to(x.dtype).cuda()).add_(0.25)
    return r, x, host(x).astype(np.float64)


def _norm_fwd_check(got, x64, res64, g64, b64, eps, dtype, what):
    y, mean, rstd, total = got
    wy, wm, wr, ws = od.layer_norm(x64, g64, b64, eps, res64)
    ab = np.abs(x64) + (np.abs(res64) if res64 is not None else 0.0)
    mb = 64 * U * ab.mean(1)                                    # error of the mean (and of s)
    _close(mean, wm, mb, "f32", what + " mean")
    # relative error of var: the deviations' own and the mean's, then the sum's
    dev = np.abs(ws - wm[:, None])
    var = (dev * dev).mean(1) + eps
    vb = (2 * (dev * (2 * U * ab + mb[:, None])).mean(1) + 64 * U * var) / var
    rb = wr * (0.6 * vb + 4 * U)
    _close(rstd, wr, rb, "f32", what + " rstd")
    gm = np.abs(g64) if g64 is not None else 1.0
    yb = gm * ((2 * U * ab + mb[:, None]) * wr[:, None] + dev * (rb + 4 * U * wr)[:, None]) + 4 * U * (
        np.abs(wy) + (np.abs(b64) if b64 is not None else 0.0))
    _close(y, wy, yb, dtype, what + " y")
    if total is not None:
        _close(total, ws, U * np.abs(ws), dtype, what + " sum")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layer_norm(d, rows, cols, dtype):
    banner(f"layer_norm {rows}x{cols} {dtype}")
    r, x, x64 = _norm_inputs(rows * 7 + cols, rows, cols, dtype, 0)
    res, res64 = _mat(r, rows, cols, 0.5, dtype)
    g, g64 = _vec(r, cols, 0.2, 1.0, dtype)
    b, b64 = _vec(r, cols, 0.2, 0.0, dtype)
    _norm_fwd_check(d.layer_norm(x, g, b, 1e-5, res), x64, res64, g64, b64, 1e-5, dtype, "norm+residual")
    got = d.layer_norm(x, g, b)
    assert got[3] is None
    _norm_fwd_check(got, x64, None, g64, b64, 1e-5, dtype, "norm")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (8, 0), (3, 0), (8, 8), (1, 3)])
def test_layer_norm_strides(d, dtype, pad, offset):
    """Rows of a wider buffer whose padding is NaN, pointers of every alignment,
    mixed parameter types, missing parameters, in-place outputs."""
    rows, cols = 21, 1000
    banner(f"layer_norm strides {dtype} {pad} {offset}")
    r, x, x64 = _norm_inputs(5, rows, cols, dtype, pad, offset)
    res, res64 = _mat(r, rows, cols, 0.5, dtype, pad, offset)
    other = "f32" if dtype == "bf16" else "bf16"
    g, g64 = _vec(r, cols, 0.2, 1.0, other)
    b, b64 = _vec(r, cols + 1, 0.2, 0.0, other)
    y, _ = _mat(r, rows, cols, 1.0, dtype, pad, offset)
    _norm_fwd_check(d.layer_norm(x, g, b[1:], 0.5, res, y=y), x64, res64, g64, b64[1:], 0.5, dtype, "strided")
    assert torch.isnan(y.as_strided((rows - 1, pad), y.stride(), y.storage_offset() + cols)).all() or pad == 0
    _norm_fwd_check(d.layer_norm(x, g, None), x64, None, g64, None, 1e-5, dtype, "no beta")
    _norm_fwd_check(d.layer_norm(x, None, b[1:]), x64, None, None, b64[1:], 1e-5, dtype, "no gamma")
    # the residual stream updated in place, the norm over x
    got = d.layer_norm(x, g, b[1:], 1e-5, res, y=x, total=res)
    assert got[0].data_ptr() == x.data_ptr() and got[3].data_ptr() == res.data_ptr()
    _norm_fwd_check(got, x64, res64, g64, b64[1:], 1e-5, dtype, "in place")


def _norm_bwd_check(got, dy64, x64, m64, r64, g64, ds64, dtype, what):
    dx, dg, db = got
    wx, wg, wb = od.layer_norm_backward(dy64, x64, m64, r64, g64, ds64)
    rows, cols = dy64.shape
    rs = r64[:, None]
    n = np.abs(x64 - m64[:, None]) * rs
    nb = 3 * U * (np.abs(x64) + np.abs(m64)[:, None]) * rs      # error of n
    g = np.abs(dy64) * (np.abs(g64) if g64 is not None else 1.0)
    c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    c2b = 64 * U * c2 + (g * nb).mean(1, keepdims=True)
    xb = rs * (4 * U * g + 66 * U * c1 + n * c2b + nb * c2 + 4 * U * n * c2) + 2 * U * (
        np.abs(ds64) if ds64 is not None else 0.0)
    _close(dx, wx, xb, dtype, what + " dx")
    # column sums: chains of rows / 512 + a joined tree of at most 512 rows
    depth = (rows / 512 + 140) * U
    if dg is not None:
        _close(dg, wg, (np.abs(dy64) * (n * depth + nb)).sum(0), "f32", what + " dgamma")
        _close(db, wb, np.abs(dy64).sum(0) * depth, "f32", what + " dbeta")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layer_norm_backward(d, rows, cols, dtype):
    banner(f"layer_norm_backward {rows}x{cols} {dtype}")
    r, x, x64 = _norm_inputs(rows * 3 + cols, rows, cols, dtype, 0)
    dy, dy64 = _mat(r, rows, cols, 0.1, dtype)
    ds, ds64 = _mat(r, rows, cols, 0.1, dtype)
    g, g64 = _vec(r, cols, 0.2, 1.0, dtype)
    _, mean, rstd, _ = od.layer_norm(x64)
    m, m64 = torch.from_numpy(mean.astype(np.float32)).cuda(), mean.astype(np.float32).astype(np.float64)
    s, s64 = torch.from_numpy(rstd.astype(np.float32)).cuda(), rstd.astype(np.float32).astype(np.float64)
    got = d.layer_norm_backward(dy, x, m, s, g, ds)
    _norm_bwd_check(got, dy64, x64, m64, s64, g64, ds64, dtype, "norm bwd+dsum")
    again = d.layer_norm_backward(dy, x, m, s, g, ds)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "equal calls give equal bits"
    _norm_bwd_check(d.layer_norm_backward(dy, x, m, s), dy64, x64, m64, s64, None, None, dtype, "norm bwd plain")
    dx, dg, db = d.layer_norm_backward(dy, x, m, s, g, need_dparams=False)
    assert dg is None and db is None
    _norm_bwd_check((dx, None, None), dy64, x64, m64, s64, g64, None, dtype, "norm bwd dx only")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1000, 40001])
def test_layer_norm_backward_strides(d, dtype, cols):
    rows = 40
    banner(f"layer_norm_backward strides {dtype} {cols}")
    r, x, x64 = _norm_inputs(11, rows, cols, dtype, 3, 1)
    dy, dy64 = _mat(r, rows, cols, 0.1, dtype, 8)
    ds, ds64 = _mat(r, rows, cols, 0.1, dtype, 1)
    g, g64 = _vec(r, cols + 1, 0.2, 1.0, "bf16")
    _, mean, rstd, _ = od.layer_norm(x64)
    m, s = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (mean, rstd))
    m64, s64 = host(m).astype(np.float64), host(s).astype(np.float64)
    got = d.layer_norm_backward(dy, x, m, s, g[1:], ds, dx=ds)
    _norm_bwd_check(got, dy64, x64, m64, s64, g64[1:], ds64, dtype, "in place over dsum")
    got = d.layer_norm_backward(dy, x, m, s, g[1:], dx=dy)
    _norm_bwd_check(got, dy64, x64, m64, s64, g64[1:], None, dtype, "in place over dy")


def test_layer_norm_of_no_rows_and_of_nan_rows(d):
    banner("layer_norm no rows")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd, _ = d.layer_norm(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    _, dg, db = d.layer_norm_backward(x, x, mean, rstd)
    assert not dg.any() and not db.any() and dg.shape == (64,)
    banner("layer_norm NaN row, constant row")
    r = np.random.default_rng(0)
    x, x64 = _mat(r, 9, 2056, 1.0, "f32")
    x[3, 100] = float("nan")
    x[5, 100] = float("inf")
    x[7] = 2.5
    y, mean, rstd, _ = d.layer_norm(x, eps=1e-6)
    ok = [0, 1, 2, 4, 6, 8]
    _norm_fwd_check((y[ok], mean[ok], rstd[ok], None), x64[ok], None, None, None, 1e-6, "f32", "rows beside NaN")
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    assert not y[7].any() and float(rstd[7]) == pytest.approx(1e3)       # no deviation: 1 / sqrt(eps)


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------

LINEAR_SHAPES = [  # M, N, K
    (1, 1, 1), (1, 7, 3), (2, 64, 8), (5, 16, 64), (16, 128, 65), (17, 130, 72), (33, 257, 128), (64, 256, 512),
    (65, 300, 515), (100, 1003, 200), (128, 128, 1024), (129, 129, 129), (200, 520, 2048), (255, 512, 88),
    (256, 256, 64), (257, 264, 56), (300, 1024, 4096), (513, 768, 320), (777, 1003, 515), (1000, 96, 1000)]
ACTS = ["none", "silu", "gelu", "relu"]


def _linear_check(y, z, x64, w64, b64, kind, res64, out, what):
    wy, wz = od.linear(x64, w64, b64, kind, res64)
    zb = 16 * U * _norms(x64, w64) + 2 * U * np.abs(wz)
    if z is not None:
        _close(z, wz, zb, out, what + " z")
    yb = 1.13 * zb + 2.0 ** -20 * np.abs(od.act(kind, wz)) + U * np.abs(wy)
    _close(y, wy, yb, out, what + " y")


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear(d, M, N, K):
    r = np.random.default_rng(M * 31 + N * 7 + K)
    x, x64 = _mat(r, M, K)
    w, w64 = _mat(r, N, K, 0.1)
    for i, out in enumerate(("bf16", "f32")):
        kind = ACTS[(M + N + K + i) % 4]
        banner(f"linear {M}x{N}x{K} {kind} {out}")
        b, b64 = _vec(r, N, 0.3, dtype=("f32", "bf16")[i])
        res, res64 = _mat(r, M, N, 1.0, out)
        y, z = d.linear(x, w, b, kind, res, DT[out], save_z=True)
        _linear_check(y, z, x64, w64, b64, kind, res64, out, f"{kind} {out}")
        y, z = d.linear(x, w, out_dtype=DT[out])
        assert z is None
        _linear_check(y, None, x64, w64, None, "none", None, out, "plain")


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M", [3, 64, 300])
def test_linear_strides(d, kind, M):
    """Rows of wider buffers (padding NaN), pointers that are not 16-byte
    aligned, strided outputs whose padding stays, the residual in place."""
    N, K = 264, 136
    r = np.random.default_rng(M)
    for pad, offset in ((0, 0), (8, 0), (8, 4), (3, 0), (1, 1)):
        for out in ("bf16", "f32"):
            banner(f"linear strides {M} {kind} {pad} {offset} {out}")
            x, x64 = _mat(r, M, K, 1.0, "bf16", pad, offset)
            w, w64 = _mat(r, N, K, 0.1, "bf16", pad, offset)
            b, b64 = _vec(r, N, 0.3)
            y, y64 = _mat(r, M, N, 1.0, out, pad, offset)
            d.linear(x, w, b, kind, residual=y, y=y)
            _linear_check(y, None, x64, w64, b64, kind, y64, out, "in place")
            if pad:
                assert torch.isnan(y.as_strided((M - 1, pad), y.stride(), y.storage_offset() + N)).all()


def test_linear_offsets_past_32_bits(d):
    """Row strides that put the last rows of x, w and y past 2^32 bytes."""
    M, N, K, ld = 700, 520, 200, 4194304
    banner("linear, offsets past 32 bits")
    r = np.random.default_rng(3)
    big = torch.zeros((M * ld,), dtype=torch.bfloat16, device="cuda")
    rows = big.view(M, ld)
    x, w, y = rows[:, :K], rows[:N, 1024:1024 + K], rows[:, 4096:4096 + N]
    x.copy_(torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)))
    w.copy_(torch.from_numpy(r.standard_normal((N, K)).astype(np.float32) * np.float32(0.1)))
    x64, w64 = host(x).astype(np.float64), host(w).astype(np.float64)
    d.linear(x, w, y=y)
    _linear_check(y, None, x64, w64, None, "none", None, "bf16", "past 32 bits")
    dy64 = host(y).astype(np.float64)
    dx, dw, _ = d.linear_backward(y, x, w, dx_dtype=torch.float32)
    _grad_check(dx, dw, None, od.linear_backward(dy64, x64, w64), dy64, x64, w64, False, "f32", "f32", "past 32 bits")


def _repeats(v, n):
    """n rows that repeat v's, on the device."""
    out = torch.empty((n,) + tuple(v.shape[1:]), dtype=v.dtype, device="cuda")
    whole = n // v.shape[0]
    out[:whole * v.shape[0]].view(whole, *v.shape).copy_(v.expand(whole, *v.shape))
    out[whole * v.shape[0]:].copy_(v[:n - whole * v.shape[0]])
    return out


def _check_repeats(got, part, what):
    """Rows of got against the checked result of the rows that they repeat:
    both within a rounding of the same sums."""
    n = part.shape[0]
    lim = 2.05 * V * part.float().abs() + 2.0 ** -16
    for r in range(0, got.shape[0], n):
        g = got[r:r + n].float()
        off = (g - part[:g.shape[0]].float()).abs() > lim[:g.shape[0]]
        assert not bool(off.any()), f"{what}: rows from {r}"
        del g, off


def test_more_rows_than_threads_of_a_launch(d):
    """Row counts whose threads would pass 2^32 in one launch."""
    banner("rows past one launch")
    r = np.random.default_rng(11)
    n = (1 << 20) + 3
    x, x64 = _mat(r, n, 8)
    g, g64 = _vec(r, 8, 0.2, 1.0)
    y, mean, rstd, _ = d.layer_norm(x, g)
    _norm_fwd_check((y, mean, rstd, None), x64, None, g64, None, 1e-5, "bf16", "part")
    rows = (1 << 26) + 7
    many = d.layer_norm(_repeats(x, rows), g)
    _check_repeats(many[0], y, "layer norm")
    _check_repeats(many[1][:, None], mean[:, None], "mean")
    del many
    w, w64 = _mat(r, 8, 8)
    y, _ = d.linear(x, w)
    _linear_check(y, None, x64, w64, None, "none", None, "bf16", "part")
    xs = _repeats(x, (1 << 30) + 77)
    out = torch.empty_like(xs)
    banner("linear of 2^30 + 77 rows")
    d.linear(xs, w, y=out)
    _check_repeats(out, y, "linear")


def _grad_check(dx, dw, db, want, dy64, x64, w64, rounded, dxt, dwt, what):
    """want: (dx, dw, dbias, dz); rounded: dz reaches the products as bf16."""
    wx, ww, wb, dz = want
    if dx is not None:
        b = 16 * U * _norms(dz, w64.T)
        if rounded:
            b = b + (4 * V + 2.0 ** -19) * np.sqrt((dz * dz) @ (w64 * w64))
        _close(dx, wx, b, dxt, what + " dx")
    if dw is not None:
        b = 16 * U * _norms(dz.T, x64.T)
        if rounded:
            b = b + (4 * V + 2.0 ** -19) * np.sqrt((dz * dz).T @ (x64 * x64))
        _close(dw, ww, b, dwt, what + " dw")
    if db is not None:
        _close(db, wb, (2.0 ** -19 + (dz.shape[0] / 256 + 100) * U) * np.abs(dz).sum(0), "f32", what + " dbias")


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear_backward(d, M, N, K):
    r = np.random.default_rng(M * 5 + N * 3 + K)
    x, x64 = _mat(r, M, K)
    w, w64 = _mat(r, N, K, 0.1)
    dy, dy64 = _mat(r, M, N, 0.1)
    for kind, zt, dxt, dwt in (("none", None, "bf16", "f32"), (ACTS[1 + (M + N + K) % 3], "bf16", "f32", "bf16"),
                               (ACTS[1 + (M + N) % 3], "f32", "bf16", "f32")):
        banner(f"linear_backward {M}x{N}x{K} {kind}")
        z, z64 = _mat(r, M, N, 1.5, zt) if zt else (None, None)
        got = d.linear_backward(dy, x, w, z, kind, DT[dxt], DT[dwt], need_dbias=True)
        _grad_check(*got, od.linear_backward(dy64, x64, w64, z64, kind), dy64, x64, w64, kind != "none", dxt, dwt, kind)
        again = d.linear_backward(dy, x, w, z, kind, DT[dxt], DT[dwt], need_dbias=True)
        assert all(torch.equal(a, b) for a, b in zip(got, again)), "equal calls give equal bits"


@pytest.mark.parametrize("kind", ["none", "gelu"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 4), (3, 0), (1, 1)])
def test_linear_backward_strides(d, kind, pad, offset):
    M, N, K = 203, 264, 136
    banner(f"linear_backward strides {kind} {pad} {offset}")
    r = np.random.default_rng(7)
    x, x64 = _mat(r, M, K, 1.0, "bf16", pad, offset)
    w, w64 = _mat(r, N, K, 0.1, "bf16", pad, offset)
    dy, dy64 = _mat(r, M, N, 0.1, "bf16", pad, offset)
    z, z64 = _mat(r, M, N, 1.5, "f32", pad, offset)
    dx, _ = _mat(r, M, K, 1.0, "bf16", pad, offset)
    dw, _ = _mat(r, N, K, 1.0, "f32", pad, offset)
    d.linear_backward(dy, x, w, z, kind, dx=dx, dw=dw)
    want = od.linear_backward(dy64, x64, w64, z64, kind)
    _grad_check(dx, dw, None, want, dy64, x64, w64, kind != "none", "bf16", "f32", "strided")
    assert torch.isnan(dx.as_strided((M - 1, pad), dx.stride(), dx.storage_offset() + K)).all()
    assert torch.isnan(dw.as_strided((N - 1, pad), dw.stride(), dw.storage_offset() + K)).all()
    # one at a time
    dx2, dw2, db2 = d.linear_backward(dy, x, w, z, kind, need_dw=False)
    assert dw2 is None and db2 is None and torch.equal(dx2, dx)
    dx3, dw3, db3 = d.linear_backward(dy, x, w, z, kind, need_dx=False)
    assert dx3 is None and torch.equal(dw3, dw)
    _, _, db4 = d.linear_backward(dy, x, w, z, kind, need_dx=False, need_dw=False, need_dbias=True)
    _grad_check(None, None, db4, want, dy64, x64, w64, True, None, None, "dbias alone")


def test_no_tokens(d):
    banner("dense operators without tokens")
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    w, w13 = e(32, 64), e(64, 48)
    y, z = d.linear(e(0, 64), w, save_z=True)
    assert y.shape == z.shape == (0, 32)
    dx, dw, db = d.linear_backward(e(0, 32), e(0, 64), w, e(0, 32), "silu", need_dbias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    a, h = d.gated_linear(e(0, 48), w13, save_h=True)
    assert a.shape == (0, 32) and h.shape == (0, 64)
    dx, dw = d.gated_linear_backward(e(0, 32), e(0, 48), w13, h)
    assert dx.shape == (0, 48) and not dw.any()


def test_linear_keeps_nan_to_its_rows_and_columns(d):
    banner("linear NaN rows")
    r = np.random.default_rng(2)
    for M, N, K in ((40, 96, 200), (300, 520, 200)):
        x, x64 = _mat(r, M, K)
        w, w64 = _mat(r, N, K, 0.1)
        x[7, 199] = float("nan")
        x[9, 0] = float("inf")
        w[33, 64] = float("nan")
        y, _ = d.linear(x, w, out_dtype=torch.float32)
        rows, cols = [i for i in range(M) if i not in (7, 9)], [i for i in range(N) if i != 33]
        assert torch.isnan(y[7]).all() and torch.isnan(y[:, 33]).all() and not torch.isfinite(y[9]).any()
        _linear_check(y[rows][:, cols], None, x64[rows], w64[cols], None, "none", None, "f32", "beside NaN")


def test_linear_on_another_stream(d):
    banner("linear on a side stream")
    r = np.random.default_rng(4)
    x, x64 = _mat(r, 300, 520)
    w, w64 = _mat(r, 264, 520, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = d.linear(x, w)
    s.synchronize()
    _linear_check(y, None, x64, w64, None, "none", None, "bf16", "side stream")


# ---------------------------------------------------------------------------
# gated linear
# ---------------------------------------------------------------------------

GATED_SHAPES = [  # M, I, H
    (1, 1, 1), (1, 16, 64), (3, 5, 9), (16, 40, 72), (17, 100, 128), (33, 128, 200), (64, 256, 512), (65, 130, 1000),
    (128, 343, 64), (200, 128, 2048), (256, 256, 256), (257, 300, 515), (333, 343, 1000), (600, 520, 136)]


def _gated_check(a, h, x64, w64, kind, out, what):
    wa, wh = od.gated_linear(x64, w64, kind)
    I = wa.shape[1]
    hb = 16 * U * _norms(x64, w64)
    if h is not None:
        _close(h, wh, hb, "bf16", what + " h")
    g, u = wh[:, :I], wh[:, I:]
    f = np.abs(od.act(kind, g))
    ab = 1.13 * hb[:, :I] * (np.abs(u) + hb[:, I:]) + f * hb[:, I:] + 2.0 ** -20 * f * np.abs(u)
    _close(a, wa, ab, out, what + " a")


@pytest.mark.parametrize("M,I,H", GATED_SHAPES)
def test_gated_linear(d, M, I, H):
    r = np.random.default_rng(M + I + H)
    x, x64 = _mat(r, M, H)
    w, w64 = _mat(r, 2 * I, H, 0.1)
    for i, out in enumerate(("bf16", "f32")):
        kind = ("silu", "gelu", "relu", "none")[(M + I + i) % 4]
        banner(f"gated_linear {M}x{I}x{H} {kind} {out}")
        a, h = d.gated_linear(x, w, kind, DT[out], save_h=True)
        _gated_check(a, h, x64, w64, kind, out, f"{kind} {out}")
        a2, h2 = d.gated_linear(x, w, kind, DT[out])
        assert h2 is None and torch.equal(a, a2)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 4), (3, 0), (1, 1)])
@pytest.mark.parametrize("M", [5, 203])
def test_gated_linear_strides(d, M, pad, offset):
    I, H = 136, 264
    banner(f"gated strides {M} {pad} {offset}")
    r = np.random.default_rng(8)
    x, x64 = _mat(r, M, H, 1.0, "bf16", pad, offset)
    w, w64 = _mat(r, 2 * I, H, 0.1, "bf16", pad, offset)
    a, _ = _mat(r, M, I, 1.0, "bf16", pad, offset)
    _, h = d.gated_linear(x, w, save_h=True, a=a)
    _gated_check(a, h, x64, w64, "silu", "bf16", "strided")
    assert torch.isnan(a.as_strided((M - 1, pad), a.stride(), a.storage_offset() + I)).all()
    da, da64 = _mat(r, M, I, 0.1, "bf16", pad, offset)
    hs, hs64 = _mat(r, M, 2 * I, 1.0, "bf16", pad, offset)
    dx, dw = d.gated_linear_backward(da, x, w, hs)
    wx, ww, dh = od.gated_linear_backward(da64, x64, w64, hs64)
    _grad_check(dx, dw, None, (wx, ww, None, dh), None, x64, w64, True, "bf16", "f32", "strided")


@pytest.mark.parametrize("M,I,H", GATED_SHAPES)
def test_gated_linear_backward(d, M, I, H):
    r = np.random.default_rng(M * 3 + I + H)
    x, x64 = _mat(r, M, H)
    w, w64 = _mat(r, 2 * I, H, 0.1)
    h, h64 = _mat(r, M, 2 * I, 1.5)
    da, da64 = _mat(r, M, I, 0.1)
    for i, (dxt, dwt) in enumerate((("bf16", "f32"), ("f32", "bf16"))):
        kind = ("silu", "gelu", "relu", "none")[(M + I + i) % 4]
        banner(f"gated_linear_backward {M}x{I}x{H} {kind}")
        dx, dw = d.gated_linear_backward(da, x, w, h, kind, DT[dxt], DT[dwt])
        wx, ww, dh = od.gated_linear_backward(da64, x64, w64, h64, kind)
        _grad_check(dx, dw, None, (wx, ww, None, dh), None, x64, w64, True, dxt, dwt, kind)
        dx2, none = d.gated_linear_backward(da, x, w, h, kind, DT[dxt], DT[dwt], need_dw=False)
        assert none is None and torch.equal(dx2, dx)


# ---------------------------------------------------------------------------
# large products, on sampled rows and columns
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(4096, 7168, 2048), (1, 7168, 2048), (32, 4096, 7168), (2048, 520, 8192),
                                   (4104, 4360, 1096)])
def test_linear_large(d, M, N, K):
    banner(f"linear {M}x{N}x{K}")
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((N, K), generator=g, device="cuda") * 0.02).bfloat16()
    dy = (torch.randn((M, N), generator=g, device="cuda") * 0.02).bfloat16()
    y, _ = d.linear(x, w, out_dtype=torch.float32)
    dx, dw, db = d.linear_backward(dy, x, w, dx_dtype=torch.float32, need_dbias=True)
    r = np.random.default_rng(0)
    rm = np.unique(np.r_[0, M - 1, r.integers(0, M, 40)])
    rn = np.unique(np.r_[0, N - 1, r.integers(0, N, 40)])
    rk = np.unique(np.r_[0, K - 1, r.integers(0, K, 40)])
    x64, w64, dy64 = host(x).astype(np.float64), host(w).astype(np.float64), host(dy).astype(np.float64)
    _linear_check(y[rm], None, x64[rm], w64, None, "none", None, "f32", "sampled rows")
    _linear_check(y[:, rn], None, x64, w64[rn], None, "none", None, "f32", "sampled columns")
    _close(dx[rm], dy64[rm] @ w64, 16 * U * _norms(dy64[rm], w64.T), "f32", "dx rows")
    _close(dx[:, rk], dy64 @ w64[:, rk], 16 * U * _norms(dy64, w64[:, rk].T), "f32", "dx columns")
    _close(dw[rn], dy64[:, rn].T @ x64, 16 * U * _norms(dy64[:, rn].T, x64.T), "f32", "dw rows")
    _close(dw[:, rk], dy64.T @ x64[:, rk], 16 * U * _norms(dy64.T, x64[:, rk].T), "f32", "dw columns")
    _close(db, dy64.sum(0), (M / 256 + 100) * U * np.abs(dy64).sum(0), "f32", "dbias")


# ---------------------------------------------------------------------------
# the sub-layer they make together
# ---------------------------------------------------------------------------

def test_dense_ffn_step(d):
    """Forward and backward of the sub-layer against the oracle's chain on the
    kernels' own saved tensors, and the gradient against differences of the
    oracle's forward."""
    T, H, I = 150, 264, 136
    banner("dense ffn step")
    r = np.random.default_rng(12)
    x, x64 = _mat(r, T, H)
    res, res64 = _mat(r, T, H)
    g, g64 = _vec(r, H, 0.1, 1.0, "bf16")
    b, b64 = _vec(r, H, 0.1, 0.0, "bf16")
    w13, w13_64 = _mat(r, 2 * I, H, 0.06)
    w2, w2_64 = _mat(r, H, I, 0.06)
    y, saved = d.dense_ffn_forward(x, g, b, w13, w2, res, training=True)
    y2, none = d.dense_ffn_forward(x, g, b, w13, w2, res)
    assert none is None and torch.equal(y, y2)
    n64, a64, s64 = (host(saved[k]).astype(np.float64) for k in ("n", "a", "s"))
    _norm_fwd_check((saved["n"], saved["mean"], saved["rstd"], saved["s"]), x64, res64, g64, b64, 1e-5, "bf16", "ffn")
    _gated_check(saved["a"], saved["h"], n64, w13_64, "silu", "bf16", "ffn")
    _linear_check(y, None, a64, w2_64, None, "none", s64, "bf16", "ffn")
    dy, dy64 = _mat(r, T, H, 0.1)
    got = d.dense_ffn_backward(dy, saved, g, w13, w2)

    def loss(x64, w13_64=w13_64, w2_64=w2_64, g64=g64):
        n, _, _, s = od.layer_norm(x64, g64, b64, 1e-5, res64)
        a, _ = od.gated_linear(n, w13_64)
        return float((od.linear(a, w2_64, residual=s)[0] * dy64).sum())

    # along random directions v, <gradient, v> is the loss's derivative; bf16
    # roundings of the activations (n, a, da, dh, dn: five of relative v each,
    # independent per element) leave the sum over many elements well inside
    # 5 v of the terms' 2-norm times a few
    for name, arr, key in (("x64", x64, "dx"), ("w13_64", w13_64, "dw13"), ("w2_64", w2_64, "dw2"), ("g64", g64, "dgamma")):
        v = r.standard_normal(arr.shape)
        base = {"x64": x64}
        up, lo = dict(base, **{name: arr + 1e-5 * v}), dict(base, **{name: arr - 1e-5 * v})
        num = (loss(**up) - loss(**lo)) / 2e-5
        terms = host(got[key]).astype(np.float64) * v
        assert abs(terms.sum() - num) <= 8 * 5 * V * np.linalg.norm(terms), (key, terms.sum(), num)


@pytest.mark.parametrize("M,I,H", [(4104, 2180, 1096), (2048, 5000, 600), (4096, 2048, 1032)])
def test_gated_linear_large(d, M, I, H):
    """Sizes of several tile shapes in one product, checked on sampled rows and
    columns (of the gate and the matching up half)."""
    banner(f"gated_linear {M}x{I}x{H}")
    g = torch.Generator(device="cuda").manual_seed(M + I)
    x = torch.randn((M, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((2 * I, H), generator=g, device="cuda") * 0.05).bfloat16()
    hs = torch.randn((M, 2 * I), generator=g, device="cuda").bfloat16()
    da = (torch.randn((M, I), generator=g, device="cuda") * 0.1).bfloat16()
    a, h = d.gated_linear(x, w, "gelu", torch.float32, save_h=True)
    dx, dw = d.gated_linear_backward(da, x, w, hs, "silu", torch.float32, torch.float32)
    r = np.random.default_rng(1)
    rm = np.unique(np.r_[0, M - 1, r.integers(0, M, 40)])
    ri = np.unique(np.r_[0, I - 1, r.integers(0, I, 40)])
    rh = np.unique(np.r_[0, H - 1, r.integers(0, H, 40)])
    both = np.r_[ri, I + ri]
    x64, w64, hs64, da64 = (host(t).astype(np.float64) for t in (x, w, hs, da))
    _gated_check(a[rm], h[rm], x64[rm], w64, "gelu", "f32", "rows")
    _gated_check(a[:, ri], h[:, both], x64, w64[both], "gelu", "f32", "columns")
    _, _, dh = od.gated_linear_backward(da64, x64, w64, hs64)
    rounded = 4 * V + 2.0 ** -19
    for got, p, q, what in ((dx[rm], dh[rm], w64, "dx rows"), (dx[:, rh], dh, w64[:, rh], "dx columns"),
                            (dw[both], dh[:, both].T, x64, "dw rows"), (dw[:, rh], dh.T, x64[:, rh], "dw columns")):
        bound = 16 * U * _norms(p, q.T) + rounded * np.sqrt((p * p) @ (q * q))
        _close(got, p @ q, bound, "f32", what)


@pytest.mark.parametrize("M,N,K", [(4096, 7168, 520), (4200, 6000, 328), (2100, 9000, 200), (8192, 1544, 264)])
def test_linear_tile_shapes(d, M, N, K):
    """Wide results that take more than one round of tiles: residual, bias and
    pre-activation over the seams between launches and shapes."""
    banner(f"linear shapes {M}x{N}x{K}")
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((N, K), generator=g, device="cuda") * 0.1).bfloat16()
    bias = torch.randn((N,), generator=g, device="cuda")
    r = np.random.default_rng(2)
    rm = np.unique(np.r_[0, M - 1, r.integers(0, M, 60)])
    x64, w64, b64 = host(x).astype(np.float64), host(w).astype(np.float64), host(bias).astype(np.float64)
    for kind, out in (("none", "bf16"), ("silu", "f32")):
        res = torch.randn((M, N), generator=g, device="cuda").to(DT[out])
        y, z = d.linear(x, w, bias, kind, res, DT[out], save_z=True)
        res64 = host(res[rm]).astype(np.float64)
        _linear_check(y[rm], z[rm], x64[rm], w64, b64, kind, res64, out, f"{kind} {out}")
        y2, _ = d.linear(x, w, bias, kind, res, DT[out])
        assert torch.equal(y, y2)


# ---------------------------------------------------------------------------
# float32 gradients where dz is formed
# ---------------------------------------------------------------------------

def _split_check(got, p, q, what):
    """A float32 product of formed dz: two bf16 terms leave at most v^2 of a
    value, each term independently, beside the float32 roundings of dz (2^-19)."""
    bound = 16 * U * _norms(p, q.T) + (4 * V * V + 2.0 ** -19) * np.sqrt((p * p) @ (q * q))
    _close(got, p @ q, bound, "f32", what)


@pytest.mark.parametrize("M,N,K", [(1, 7, 3), (33, 257, 128), (65, 300, 515), (513, 768, 320), (3000, 130, 72)])
def test_float32_gradients_of_an_activation(d, M, N, K):
    r = np.random.default_rng(M + N)
    x, x64 = _mat(r, M, K)
    w, w64 = _mat(r, N, K, 0.1)
    dy, dy64 = _mat(r, M, N, 0.1)
    for kind in ("silu", "gelu"):
        banner(f"float32 gradients of {kind}, {M}x{N}x{K}")
        z, z64 = _mat(r, M, N, 1.5)
        dz = od.linear_backward(dy64, x64, w64, z64, kind)[3]
        dx, dw, _ = d.linear_backward(dy, x, w, z, kind, torch.float32, torch.float32)
        _split_check(dx, dz, w64, "dx")
        _split_check(dw, dz.T, x64, "dw")
        again = d.linear_backward(dy, x, w, z, kind, torch.float32, torch.float32)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("M,I,H", [(1, 1, 1), (3, 5, 9), (65, 130, 1000), (333, 343, 1000), (2000, 520, 136),
                                   (538, 2316, 5156)])   # dw in two launches
def test_float32_gradients_of_a_gated_product(d, M, I, H):
    r = np.random.default_rng(M + I)
    x, x64 = _mat(r, M, H)
    w, w64 = _mat(r, 2 * I, H, 0.1)
    h, h64 = _mat(r, M, 2 * I, 1.5)
    da, da64 = _mat(r, M, I, 0.1)
    for kind in ("silu", "none"):
        banner(f"float32 gradients of gated {kind}, {M}x{I}x{H}")
        dh = od.gated_linear_backward(da64, x64, w64, h64, kind)[2]
        dx, dw = d.gated_linear_backward(da, x, w, h, kind, torch.float32, torch.float32)
        _split_check(dx, dh, w64, "dx")
        _split_check(dw, dh.T, x64, "dw13")
        # one gradient of each type, and one alone
        dx16, dw32 = d.gated_linear_backward(da, x, w, h, kind)
        assert torch.equal(dw32, dw)
        _grad_check(dx16, None, None, (dh @ w64, None, None, dh), None, x64, w64, True, "bf16", None, "dx bf16")
        assert torch.equal(d.gated_linear_backward(da, x, w, h, kind, need_dx=False)[1], dw)


def test_bf16_dz_on_request_and_infinite_dz(d):
    banner("dz_dtype bf16; infinite dz")
    M, N, K = 300, 264, 136
    r = np.random.default_rng(6)
    x, x64 = _mat(r, M, K)
    w, w64 = _mat(r, N, K, 0.1)
    dy, dy64 = _mat(r, M, N, 0.1)
    z, z64 = _mat(r, M, N, 1.5)
    f32, b16 = torch.float32, torch.bfloat16
    got = d.linear_backward(dy, x, w, z, "silu", f32, f32, need_dbias=True, dz_dtype=b16)
    _grad_check(*got, od.linear_backward(dy64, x64, w64, z64, "silu"), dy64, x64, w64, True, "f32", "f32", "bf16 dz")
    full = d.linear_backward(dy, x, w, z, "silu", f32, f32, need_dbias=True)
    assert not torch.equal(got[1], full[1]) and torch.equal(got[2], full[2])
    # bf16 gradients and exact products are the same either way
    for act, zz, dt in (("silu", z, b16), ("none", None, f32)):
        a, b = (d.linear_backward(dy, x, w, zz, act, dt, dt, dz_dtype=t) for t in (None, b16))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    h, h64 = _mat(r, M, 2 * N, 1.5)
    w13, w13_64 = _mat(r, 2 * N, K, 0.1)
    gx, gw = d.gated_linear_backward(dy, x, w13, h, "gelu", f32, f32, dz_dtype=b16)
    wx, ww, dh = od.gated_linear_backward(dy64, x64, w13_64, h64, "gelu")
    _grad_check(gx, gw, None, (wx, ww, None, dh), None, x64, w13_64, True, "f32", "f32", "gated bf16 dz")
    # an infinity in dz is one in the products, not the NaN of its rounding's rest
    dy[5, 7] = float("inf")
    z[5, 7] = 1.0
    dx, dw, _ = d.linear_backward(dy, x, w, z, "silu", f32, f32)
    assert torch.isinf(dx[5]).all() and torch.isinf(dw[7]).all()
    rows, cols = [i for i in range(M) if i != 5], [i for i in range(N) if i != 7]
    assert torch.isfinite(dx[rows]).all() and torch.isfinite(dw[cols]).all()
    need = d.linear_backward_workspace_bytes(dy, x, w, "silu")
    assert need > d.linear_backward_workspace_bytes(dy, x, w, "silu", b16)
    with pytest.raises(TypeError):
        d.linear_backward(dy, x, w, z, "silu", dz_dtype=torch.float16)


# ---------------------------------------------------------------------------
# activations at exact arguments
# ---------------------------------------------------------------------------

# z of either sign from the smallest normal float to past where e^z and the
# normal distribution's tail leave float32's range
_Z = np.sort(np.concatenate([s * np.concatenate([np.linspace(0.0, 16.0, 3001), np.linspace(16.0, 120.0, 1000),
                                                 2.0 ** np.linspace(-126, 0, 300)]) for s in (1.0, -1.0)]).astype(np.float32))


def _act_terms(kind, z):
    """(act, |terms of act'| summed, act') in float64, no difference of near values."""
    if kind == "relu":
        return np.maximum(z, 0.0), (z > 0) * 1.0, (z > 0) * 1.0
    if kind == "silu":
        p, q = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
        return z * p, p * (1.0 + np.abs(z) * q), p * (1.0 + z * q)
    phi = 0.5 * np.array([math.erfc(-v / math.sqrt(2.0)) for v in z])
    pdf = np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return z * phi, phi + np.abs(z) * pdf, phi + z * pdf


@pytest.mark.parametrize("tokens", [1, 80])
@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_activation_at_exact_arguments(d, kind, tokens):
    """act and act' within 2^-20 of their value (of the sum of act's two terms'
    sizes, which cancel at its zero), where float32 has one: z = bias exactly,
    as x = 0, and the bias gradient of one row of ones is act'(z)."""
    banner(f"activation {kind} {tokens}")
    z64 = _Z.astype(np.float64)
    n = z64.size
    z = torch.from_numpy(_Z).cuda()
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    tiny = 2.0 ** -126
    f, terms, df = _act_terms(kind, z64)
    y, saved = d.linear(e(tokens, 8), e(n, 8), z, kind, out_dtype=torch.float32, save_z=True)
    assert torch.equal(saved, z.expand(tokens, n))
    _close(y, np.broadcast_to(f, (tokens, n)), 2.0 ** -20 * np.abs(f) + tiny, "f32", f"{kind}")
    _, _, db = d.linear_backward(e(1, n) + 1, e(1, 8), e(n, 8), z[None], kind, need_dx=False, need_dw=False,
                                 need_dbias=True)
    _close(db, df, 2.0 ** -20 * terms + tiny, "f32", f"{kind}'")
    # the gate of the gated product: g exact (one product with 1), u = 1
    g = z.bfloat16()
    g64 = host(g).astype(np.float64)
    f, terms, df = _act_terms(kind, g64)
    one = e(tokens, 1) + 1
    w13 = torch.cat([g[:, None], torch.ones_like(g)[:, None]])
    a, h = d.gated_linear(one, w13, kind, torch.float32, save_h=True)
    assert torch.equal(h[0], w13[:, 0])
    _close(a, np.broadcast_to(f, (tokens, n)), 2.0 ** -20 * np.abs(f) + tiny, "f32", f"gated {kind}")


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_activation_of_infinities_and_nan(d, kind):
    """As in the formulas: z / (1 + e^-z) and z (1 + erf) / 2 at minus infinity
    are infinity times 0, max(z, 0) is 0."""
    banner(f"activation {kind}, infinities")
    z = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0], device="cuda")
    x, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 8), (4, 8)))
    y = host(d.linear(x, w, z, kind, out_dtype=torch.float32)[0])[0]
    assert y[0] == np.inf and np.isnan(y[2]) and np.isfinite(y[3])
    assert y[1] == 0 if kind == "relu" else np.isnan(y[1])
