"""The routed experts' feed-forward pass outside FP8, over the calls of
include/dsmoe_experts.h: grouped_linear and grouped_gated_linear in bf16 with
their backward passes, int8_linear and int8_gated_linear on 8-bit integers, and
the experts' whole pass that they make with the routing and the combine.

Matrices are 2-D with contiguous columns; rows may be strided (a slice of a
wider buffer).  Weights of G experts are 3-D, [G][N][K], a matrix of all their
rows.  offsets int32 [G+1] on the device says which rows are whose (None: all
rows are those of one expert), rows int32 [R] which row of the source a row is
(None: itself).  Outputs that are not passed in are allocated; their rows outside
every group are not written.  As everywhere in this package the wrappers check
types, devices and shapes, marshal the arguments and launch on the current
stream.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import BF16, F32, _dtype_code, combine_rows, lib
from .dense import (_MAT, _act, _begin, _check, _declare, _grad_act, _i64, _int, _mat, _new, _out, _scratch, _sz,
                    _vec, _vp)

__all__ = ["grouped_linear", "grouped_linear_backward", "grouped_gated_linear", "grouped_gated_linear_backward",
           "router_backward", "quant_rows_int8", "int8_linear", "int8_gated_linear", "moe_ffn_forward",
           "moe_ffn_backward", "moe_ffn_int8_forward"]

_ROWS = [_vp, _i64, _i64, _vp]            # matrix, its rows, index
_SROWS = [_vp, _i64, _vp, _i64, _vp]      # matrix, scales, its rows, index
_i32 = _int

_declare("dsmoe_grouped_linear_workspace_bytes", _sz, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_grouped_linear", _int, _ROWS, _MAT, _vp, _i32, _i64, _i64, _i64, _MAT, _int, _vp, _sz, _vp)
_declare("dsmoe_grouped_linear_backward_workspace_bytes", _sz, _ROWS, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_grouped_linear_backward", _int, _ROWS, _ROWS, _MAT, _vp, _i32, _i64, _i64, _i64, _MAT, _int, _MAT,
         _int, _vp, _sz, _vp)
_declare("dsmoe_grouped_gated_linear_workspace_bytes", _sz, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_grouped_gated_linear", _int, _ROWS, _MAT, _vp, _int, _vp, _i32, _i64, _i64, _i64, _MAT, _int, _MAT,
         _vp, _sz, _vp)
_declare("dsmoe_grouped_gated_linear_backward_workspace_bytes", _sz, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_grouped_gated_linear_backward", _int, _MAT, _ROWS, _MAT, _MAT, _vp, _int, _vp, _i32, _i64, _i64, _i64,
         _MAT, _int, _MAT, _int, _vp, _vp, _sz, _vp)
_declare("dsmoe_router_backward", _int, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp)
_declare("dsmoe_quant_rows_int8", _int, _MAT, _int, _i64, _i64, _MAT, _vp, _vp)
_declare("dsmoe_int8_linear_workspace_bytes", _sz, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_int8_linear", _int, _SROWS, _MAT, _vp, _vp, _i32, _i64, _i64, _i64, _MAT, _int, _vp, _sz, _vp)
_declare("dsmoe_int8_gated_linear_workspace_bytes", _sz, _ROWS, _MAT, _i32, _i64, _i64, _i64)
_declare("dsmoe_int8_gated_linear", _int, _SROWS, _MAT, _vp, _vp, _int, _vp, _i32, _i64, _i64, _i64, _MAT, _int, _vp,
         _sz, _vp)

EXPORTED_EXPERTS = (
    "dsmoe_grouped_linear_workspace_bytes", "dsmoe_grouped_linear", "dsmoe_grouped_linear_backward_workspace_bytes",
    "dsmoe_grouped_linear_backward", "dsmoe_grouped_gated_linear_workspace_bytes", "dsmoe_grouped_gated_linear",
    "dsmoe_grouped_gated_linear_backward_workspace_bytes", "dsmoe_grouped_gated_linear_backward",
    "dsmoe_router_backward", "dsmoe_quant_rows_int8", "dsmoe_int8_linear_workspace_bytes", "dsmoe_int8_linear",
    "dsmoe_int8_gated_linear_workspace_bytes", "dsmoe_int8_gated_linear")


def _experts(t, dtype, name, device):
    """(pointer, row stride, G, N, K) of the weights of G experts."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [experts][rows][columns]")
    G, N, K = t.shape
    gs, ld, cs = t.stride()
    if K > 1 and cs != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if N == 1:
        ld = gs if G > 1 else K
    elif G > 1 and gs != N * ld:
        raise ValueError(f"the experts of {name} must follow one another as the rows of one matrix")
    if G * N > 1 and ld < K:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), ld, G, N, K


def _experts_out(t, G, N, K, dtype, name, device):
    """(tensor, pointer, row stride, dtype code) of weight gradients."""
    if t is None:
        t = torch.empty((G, N, K), dtype=dtype, device=device)
        return t, t.data_ptr(), K, _dtype_code(dtype)
    p, ld, g, n, k = _experts(t, t.dtype, name, device)
    if (g, n, k) != (G, N, K):
        raise ValueError(f"{name} must be {[G, N, K]}, got {list(t.shape)}")
    return t, p, ld, _dtype_code(t.dtype)


def _offsets(t, G, device):
    if t is None:
        if G != 1:
            raise ValueError("offsets may be None only for one expert")
        return None
    return _int_vec(t, G + 1, "offsets", device)


def _int_vec(t, n, name, device):
    """Pointer of a contiguous int32 vector of n values (None: any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or (t.shape[0] > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector" + ("" if n is None else f" of {n} values"))
    return t.data_ptr()


def _rows(t, x, name, device, R=None):
    """(pointer, number of rows) of the index of x's rows; R: the number that
    there must be."""
    if t is None:
        if R is not None and x.shape[0] != R:
            raise ValueError(f"{x.shape[0]} rows where {R} are expected")
        return None, x.shape[0]
    return _int_vec(t, R, name, device), t.shape[0]


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                   rows: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, y: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """y[r] = x[rows[r]] W_g^T for the rows r of each expert g
    (dsmoe_grouped_linear).  x bf16 [n][K], w bf16 [G][N][K].  Returns y [R][N]
    (bf16 or f32)."""
    device, stream = _begin(x, "x")
    xp, ldx = _mat(x, None, torch.bfloat16, "x")
    wp, ldw, G, N, K = _experts(w, torch.bfloat16, "w", device)
    if x.shape[1] != K:
        raise ValueError("x and w must have the same K")
    op = _offsets(offsets, G, device)
    ip, R = _rows(rows, x, "rows", device)
    y, yp, ldy = _out(y, R, N, out_dtype, "y", device)
    yt = _dtype_code(y.dtype)
    n = x.shape[0]
    need = lib.dsmoe_grouped_linear_workspace_bytes(xp, ldx, n, ip, wp, ldw, G, R, N, K) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_grouped_linear(xp, ldx, n, ip, wp, ldw, op, G, R, N, K, yp, ldy, yt, sp, sn, stream),
           "dsmoe_grouped_linear")
    return y


def grouped_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                            rows: Optional[torch.Tensor] = None, dy_rows: Optional[torch.Tensor] = None,
                            dx_dtype=torch.bfloat16, dw_dtype=torch.float32, need_dx: bool = True,
                            need_dw: bool = True, dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Gradients of grouped_linear (dsmoe_grouped_linear_backward).  dy bf16
    [n_dy][N], row r being dy[dy_rows[r]] (the gradient of the layer's output, by
    token); x, w, rows the forward's.  Returns (dx [R][K], one row per routed
    row, dw [G][N][K]), None where not wanted."""
    device, stream = _begin(dy, "dy")
    dyp, lddy = _mat(dy, None, torch.bfloat16, "dy")
    wp, ldw, G, N, K = _experts(w, torch.bfloat16, "w", device)
    if dy.shape[1] != N:
        raise ValueError("dy and w must have the same N")
    xp, ldx = _mat(x, None, torch.bfloat16, "x", device)
    if x.shape[1] != K:
        raise ValueError("x and w must have the same K")
    op = _offsets(offsets, G, device)
    dip, R = _rows(dy_rows, dy, "dy_rows", device)
    ip, _ = _rows(rows, x, "rows", device, R)
    dxp, lddx, dxt, dwp, lddw, dwt = None, 0, BF16, None, 0, F32
    if dx is not None or need_dx:
        dx, dxp, lddx = _out(dx, R, K, dx_dtype, "dx", device)
        dxt = _dtype_code(dx.dtype)
    if dw is not None or need_dw:
        dw, dwp, lddw, dwt = _experts_out(dw, G, N, K, dw_dtype, "dw", device)
    nd, n = dy.shape[0], x.shape[0]
    need = lib.dsmoe_grouped_linear_backward_workspace_bytes(dyp, lddy, nd, dip, xp, ldx, n, ip, wp, ldw, G, R, N, K) \
        if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_grouped_linear_backward(dyp, lddy, nd, dip, xp, ldx, n, ip, wp, ldw, op, G, R, N, K, dxp, lddx,
                                             dxt, dwp, lddw, dwt, sp, sn, stream), "dsmoe_grouped_linear_backward")
    return dx, dw


def grouped_gated_linear(x: torch.Tensor, w13: torch.Tensor, offsets: Optional[torch.Tensor], act: str = "silu",
                         rows: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
                         out_dtype=torch.bfloat16, save_h: bool = False, a: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """a[r] = row_scale[r] act(x[rows[r]] Wg_g^T) * (x[rows[r]] Wu_g^T) with w13
    = [Wg; Wu] of each expert g (dsmoe_grouped_gated_linear).  x bf16 [n][H],
    w13 bf16 [G][2I][H], row_scale f32 [R] (the rows' gates).  Returns (a
    [R][I], h): h = [g | u] bf16 [R][2I] with save_h, else None."""
    device, stream = _begin(x, "x")
    code = _act(act)
    xp, ldx = _mat(x, None, torch.bfloat16, "x")
    wp, ldw, G, N2, H = _experts(w13, torch.bfloat16, "w13", device)
    I = N2 // 2
    if x.shape[1] != H or N2 != 2 * I:
        raise ValueError("w13 must be [experts][2I][H] with x's H")
    op = _offsets(offsets, G, device)
    ip, R = _rows(rows, x, "rows", device)
    gp, _ = _vec(row_scale, R, "row_scale", device, torch.float32)
    a, ap, lda = _out(a, R, I, out_dtype, "a", device)
    at = _dtype_code(a.dtype)
    h, hp, ldh = _new(R, N2, torch.bfloat16, device) if save_h else (None, None, 0)
    n = x.shape[0]
    need = lib.dsmoe_grouped_gated_linear_workspace_bytes(xp, ldx, n, ip, wp, ldw, G, R, H, I) \
        if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_grouped_gated_linear(xp, ldx, n, ip, wp, ldw, gp, code, op, G, R, H, I, ap, lda, at, hp, ldh, sp,
                                          sn, stream), "dsmoe_grouped_gated_linear")
    return a, h


def grouped_gated_linear_backward(da: torch.Tensor, x: torch.Tensor, w13: torch.Tensor, h: torch.Tensor,
                                  offsets: Optional[torch.Tensor], act: str = "silu",
                                  rows: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
                                  dx_dtype=torch.bfloat16, dw_dtype=torch.float32, need_dx: bool = True,
                                  need_dw: bool = True, need_dscale: bool = False, dx: Optional[torch.Tensor] = None,
                                  dw13: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                  dz_dtype: Optional[torch.dtype] = None):
    """Gradients of grouped_gated_linear (dsmoe_grouped_gated_linear_backward)
    from the saved h.  da bf16 [R][I].  Float32 gradients keep 16 bits of the
    gradient at h by a second product, which takes longer than the first, as it
    reads the result back; dz_dtype torch.bfloat16 rounds it to bf16 for them too,
    as for bf16 gradients, whose error is then 1.4 times their own rounding's (a
    float32 gradient that is rounded afterwards has only that).  Returns (dx [R][H], one row per
    routed row, dw13 [G][2I][H], dscale f32 [R]), None where not wanted."""
    device, stream = _begin(da, "da")
    code = _grad_act(act, dz_dtype)
    dap, ldda = _mat(da, None, torch.bfloat16, "da")
    R, I = da.shape
    wp, ldw, G, N2, H = _experts(w13, torch.bfloat16, "w13", device)
    xp, ldx = _mat(x, None, torch.bfloat16, "x", device)
    if N2 != 2 * I or x.shape[1] != H:
        raise ValueError("w13 must be [experts][2I][H] with da's I and x's H")
    hp, ldh = _mat(h, (R, N2), torch.bfloat16, "h", device)
    op = _offsets(offsets, G, device)
    ip, _ = _rows(rows, x, "rows", device, R)
    gp, _ = _vec(row_scale, R, "row_scale", device, torch.float32)
    dxp, lddx, dxt, dwp, lddw, dwt = None, 0, BF16, None, 0, F32
    if dx is not None or need_dx:
        dx, dxp, lddx = _out(dx, R, H, dx_dtype, "dx", device)
        dxt = _dtype_code(dx.dtype)
    if dw13 is not None or need_dw:
        dw13, dwp, lddw, dwt = _experts_out(dw13, G, N2, H, dw_dtype, "dw13", device)
    dscale = torch.empty((R,), dtype=torch.float32, device=device) if need_dscale else None
    n = x.shape[0]
    need = lib.dsmoe_grouped_gated_linear_backward_workspace_bytes(xp, ldx, n, ip, wp, ldw, G, R, H, I) \
        if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_grouped_gated_linear_backward(
        dap, ldda, xp, ldx, n, ip, wp, ldw, hp, ldh, gp, code, op, G, R, H, I, dxp, lddx, dxt, dwp, lddw, dwt,
        None if dscale is None else dscale.data_ptr(), sp, sn, stream), "dsmoe_grouped_gated_linear_backward")
    return dx, dw13, dscale


def router_backward(dgate: torch.Tensor, topk_idx: torch.Tensor, logits: torch.Tensor):
    """Gradients of the router logits (dsmoe_router_backward) from those of the
    gates, f32 [T][K]; topk_idx int32 [T][K], logits f32 [T][E].  Returns dlogits
    f32 [T][E]."""
    device, stream = _begin(logits, "logits")
    for t, dtype, name in ((dgate, torch.float32, "dgate"), (topk_idx, torch.int32, "topk_idx"),
                           (logits, torch.float32, "logits")):
        if t.device != device or t.dtype != dtype or t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} matrix on {device}")
    (T, E), K = logits.shape, topk_idx.shape[1]
    if topk_idx.shape[0] != T or dgate.shape != topk_idx.shape:
        raise ValueError("dgate and topk_idx must be [T][K] with logits' T")
    dlogits = torch.empty_like(logits)
    _check(lib.dsmoe_router_backward(dgate.data_ptr(), topk_idx.data_ptr(), logits.data_ptr(), T, E, K,
                                     dlogits.data_ptr(), stream), "dsmoe_router_backward")
    return dlogits


def quant_rows_int8(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """8-bit integers with one scale per row (dsmoe_quant_rows_int8).  x bf16 or
    f32, [rows][cols] or the weights of experts [G][N][K].  Returns (q int8 like
    x, scale f32 [rows] or [G][N])."""
    device, stream = _begin(x, "x")
    xt = _dtype_code(x.dtype)
    if x.dim() == 3:
        xp, ldx, G, N, cols = _experts(x, x.dtype, "x", device)
        rows = G * N
    else:
        xp, ldx = _mat(x, None, None, "x")
        rows, cols = x.shape
    if q is None:
        q = torch.empty(x.shape, dtype=torch.int8, device=device)
        qp, ldq = q.data_ptr(), cols
    elif q.shape != x.shape:
        raise ValueError("q must have x's shape")
    elif x.dim() == 3:
        qp, ldq = _experts(q, torch.int8, "q", device)[:2]
    else:
        qp, ldq = _mat(q, None, torch.int8, "q", device)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    elif scale.shape != x.shape[:-1] or scale.dtype != torch.float32 or scale.device != device \
            or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor of x's rows")
    _check(lib.dsmoe_quant_rows_int8(xp, ldx, xt, rows, cols, qp, ldq, scale.data_ptr(), stream),
           "dsmoe_quant_rows_int8")
    return q, scale


def _int8_operands(x, x_scale, w, w_scale, offsets, rows):
    """Pointers and sizes of an 8-bit product."""
    device, stream = _begin(x, "x")
    xp, ldx = _mat(x, None, torch.int8, "x")
    wp, ldw, G, N, K = _experts(w, torch.int8, "w", device)
    if x.shape[1] != K:
        raise ValueError("x and w must have the same row length")
    xsp, _ = _vec(x_scale, x.shape[0], "x_scale", device, torch.float32)
    if not isinstance(w_scale, torch.Tensor) or w_scale.device != device or w_scale.dtype != torch.float32 \
            or not w_scale.is_contiguous() or w_scale.shape != w.shape[:-1]:
        raise ValueError("w_scale must be a contiguous float32 tensor of w's rows")
    op = _offsets(offsets, G, device)
    ip, R = _rows(rows, x, "rows", device)
    return device, stream, (xp, ldx, x.shape[0], ip), xsp, (wp, ldw), w_scale.data_ptr(), op, G, N, K, R


def int8_linear(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                offsets: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                out_dtype=torch.bfloat16, y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """y[r][c] = x_scale[rows[r]] w_scale[g][c] (x[rows[r]] . w[g][c]) on 8-bit
    integers (dsmoe_int8_linear).  x int8 [n][K] with x_scale f32 [n], w int8
    [G][N][K] with w_scale f32 [G][N], as from quant_rows_int8; without offsets
    one expert's, also as [N][K] with [N]: a dense product.  Returns y [R][N]
    (bf16 or f32)."""
    device, stream, (xp, ldx, n, ip), xsp, (wp, ldw), wsp, op, G, N, K, R = _int8_operands(x, x_scale, w, w_scale,
                                                                                          offsets, rows)
    y, yp, ldy = _out(y, R, N, out_dtype, "y", device)
    yt = _dtype_code(y.dtype)
    need = lib.dsmoe_int8_linear_workspace_bytes(xp, ldx, n, ip, wp, ldw, G, R, N, K) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_int8_linear(xp, ldx, xsp, n, ip, wp, ldw, wsp, op, G, R, N, K, yp, ldy, yt, sp, sn, stream),
           "dsmoe_int8_linear")
    return y


def int8_gated_linear(x: torch.Tensor, x_scale: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, act: str = "silu", rows: Optional[torch.Tensor] = None,
                      row_scale: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                      a: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """grouped_gated_linear on 8-bit integers (dsmoe_int8_gated_linear): x int8
    [n][H] with x_scale f32 [n], w13 int8 [G][2I][H] with w13_scale f32 [G][2I].
    Returns a [R][I] (bf16 or f32)."""
    code = _act(act)
    device, stream, (xp, ldx, n, ip), xsp, (wp, ldw), wsp, op, G, N2, H, R = _int8_operands(x, x_scale, w13, w13_scale,
                                                                                           offsets, rows)
    I = N2 // 2
    if N2 != 2 * I:
        raise ValueError("w13 must be [experts][2I][H]")
    gp, _ = _vec(row_scale, R, "row_scale", device, torch.float32)
    a, ap, lda = _out(a, R, I, out_dtype, "a", device)
    at = _dtype_code(a.dtype)
    need = lib.dsmoe_int8_gated_linear_workspace_bytes(xp, ldx, n, ip, wp, ldw, G, R, H, I) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_int8_gated_linear(xp, ldx, xsp, n, ip, wp, ldw, wsp, gp, code, op, G, R, H, I, ap, lda, at, sp, sn,
                                       stream), "dsmoe_int8_gated_linear")
    return a


def _tokens(x, routing):
    """x and the routing are of the same tokens."""
    if x.shape[0] != routing["inv"].shape[0]:
        raise ValueError(f"x has {x.shape[0]} tokens, the routing {routing['inv'].shape[0]}")


def _routed_rows(routing, n_shared):
    """(offsets, tokens of the rows, gates of the rows, first shared row or -1):
    the routed rows and, with a shared expert, one more group of every token
    with gate 1."""
    if n_shared not in (0, 1):
        raise ValueError("n_shared must be 0 or 1")
    off, perm, inv, gates = (routing[k] for k in ("offsets", "perm", "inv", "gates"))
    T, routed = inv.shape[0], perm.numel()
    scale = torch.ones((routed + n_shared * T,), dtype=torch.float32, device=perm.device)
    scale[inv.reshape(-1).long()] = gates.reshape(-1)
    if n_shared:
        off = torch.cat([off, torch.full((1,), routed + T, dtype=torch.int32, device=perm.device)])
        perm = torch.cat([perm, torch.arange(T, dtype=torch.int32, device=perm.device)])
    return off, perm, scale, routed if n_shared else -1


def moe_ffn_forward(x: torch.Tensor, routing: dict, w13: torch.Tensor, w2: torch.Tensor, act: str = "silu",
                    n_shared: int = 0, training: bool = False, out_dtype=torch.bfloat16):
    """The experts' feed-forward pass in bf16:

        y[t] = sum over the experts e of token t of
               gate[t, e] (act(x[t] Wg_e^T) * (x[t] Wu_e^T)) W2_e^T

    x bf16 [T][H], routing as from route(); w13 bf16 [E][2I][H], w2 bf16
    [E][H][I], with n_shared = 1 one more expert that every token takes with
    gate 1.  H is a multiple of 8, E + n_shared at most 1024.  out_dtype is the
    type of y and of the terms that the sum over the experts adds up in float32:
    in bf16 each is rounded on the way, as y is at the end, which saves half of
    their bytes; float32 (as the FP8 layer's) rounds neither.  Returns (y, saved):
    y [T][H] and, when training, what moe_ffn_backward needs."""
    off, perm, scale, shared0 = _routed_rows(routing, n_shared)
    _tokens(x, routing)
    a, h = grouped_gated_linear(x, w13, off, act, rows=perm, row_scale=scale, save_h=training)
    o = grouped_linear(a, w2, off, out_dtype=out_dtype)
    y = combine_rows(o, routing["inv"], shared0)
    return y, ({"offsets": off, "perm": perm, "scale": scale, "shared0": shared0, "a": a, "h": h} if training else None)


def moe_ffn_backward(dy: torch.Tensor, x: torch.Tensor, routing: dict, w13: torch.Tensor, w2: torch.Tensor,
                     saved: dict, act: str = "silu", logits: Optional[torch.Tensor] = None, dw_dtype=torch.float32,
                     dz_dtype: Optional[torch.dtype] = None, dx_dtype=torch.bfloat16):
    """Gradients of moe_ffn_forward from dy bf16 [T][H] and its saved dict;
    dz_dtype as in grouped_gated_linear_backward; dx_dtype the type of dx and of
    the terms that its sum over a token's experts adds up, as out_dtype of the
    forward.  The gradient at the activations is bf16, as the operand of what
    follows.  Returns {"dx" [T][H], "dw13", "dw2", "dgates" f32 [T][K]} and, with
    the router logits f32 [T][E], "dlogits" (the routing held fixed)."""
    off, perm, inv = saved["offsets"], saved["perm"], routing["inv"]
    if dy.shape != x.shape or x.shape[0] != inv.shape[0]:
        raise ValueError("dy and x must be [T][H] with the routing's T")
    da, dw2 = grouped_linear_backward(dy, saved["a"], w2, off, dy_rows=perm, dw_dtype=dw_dtype)
    dx_rows, dw13, dscale = grouped_gated_linear_backward(da, x, w13, saved["h"], off, act, rows=perm,
                                                          row_scale=saved["scale"], dx_dtype=dx_dtype,
                                                          dw_dtype=dw_dtype, need_dscale=True, dz_dtype=dz_dtype)
    out = {"dx": combine_rows(dx_rows, inv, saved["shared0"]), "dw13": dw13, "dw2": dw2, "dgates": dscale[inv.long()]}
    if logits is not None:
        out["dlogits"] = router_backward(out["dgates"], routing["topk_idx"], logits)
    return out


def moe_ffn_int8_forward(x: torch.Tensor, routing: dict, w13: tuple, w2: tuple, act: str = "silu", n_shared: int = 0,
                         out_dtype=torch.bfloat16):
    """moe_ffn_forward on 8-bit integers: w13 and w2 are (codes, scales) of the
    experts' weights as from quant_rows_int8; x and the activations are
    quantised per row on the way.  x bf16 [T][H]; returns y [T][H]."""
    off, perm, scale, shared0 = _routed_rows(routing, n_shared)
    _tokens(x, routing)
    q, s = quant_rows_int8(x)
    a = int8_gated_linear(q, s, *w13, off, act, rows=perm, row_scale=scale)
    q, s = quant_rows_int8(a)
    return combine_rows(int8_linear(q, s, *w2, off, out_dtype=out_dtype), routing["inv"], shared0)
