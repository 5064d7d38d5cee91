"""The dense (not routed) feed-forward sub-layer beside the MoE layer, in
bf16: layer_norm, gated_linear and linear with their backward passes, over
the calls of include/dsmoe_dense.h, and the sub-layer they make together.

Matrices are 2-D with contiguous columns; rows may be strided (a slice of a
wider buffer).  Outputs that are not passed in are allocated.  As everywhere
in this package the wrappers check types, devices and shapes, marshal the
arguments and launch on the current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import BF16, F32, DsmoeError, _dtype_code, lib

__all__ = ["ACTIVATIONS", "layer_norm", "layer_norm_backward", "linear", "linear_backward", "gated_linear",
           "gated_linear_backward", "dense_ffn_forward", "dense_ffn_backward"]

# dsmoe_act codes
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
# DSMOE_DZ_BF16
_DZ_BF16 = 16

_vp, _i64, _int, _sz, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_MAT = [_vp, _i64]


def _declare(name, restype, *argtypes):
    f = getattr(lib, name)
    f.restype = restype
    f.argtypes = [a for t in argtypes for a in (t if isinstance(t, list) else [t])]


_declare("dsmoe_layer_norm", _int, _MAT, _MAT, _int, _vp, _vp, _int, _i64, _i64, _f32, _MAT, _MAT, _vp, _vp, _vp)
_declare("dsmoe_layer_norm_backward_workspace_bytes", _sz, _i64, _i64)
_declare("dsmoe_layer_norm_backward", _int, _MAT, _MAT, _MAT, _int, _vp, _int, _vp, _vp, _i64, _i64, _MAT, _vp, _vp,
         _vp, _sz, _vp)
_declare("dsmoe_linear_workspace_bytes", _sz, _MAT, _MAT, _i64, _i64, _i64)
_declare("dsmoe_linear", _int, _MAT, _MAT, _vp, _int, _MAT, _int, _i64, _i64, _i64, _MAT, _int, _MAT, _vp, _sz, _vp)
_declare("dsmoe_linear_backward_workspace_bytes", _sz, _MAT, _MAT, _MAT, _int, _i64, _i64, _i64)
_declare("dsmoe_linear_backward", _int, _MAT, _MAT, _MAT, _MAT, _int, _int, _i64, _i64, _i64, _MAT, _int, _MAT, _int,
         _vp, _vp, _sz, _vp)
_declare("dsmoe_gated_linear_workspace_bytes", _sz, _MAT, _MAT, _i64, _i64, _i64)
_declare("dsmoe_gated_linear", _int, _MAT, _MAT, _int, _i64, _i64, _i64, _MAT, _int, _MAT, _vp, _sz, _vp)
_declare("dsmoe_gated_linear_backward_workspace_bytes", _sz, _MAT, _MAT, _i64, _i64, _i64)
_declare("dsmoe_gated_linear_backward", _int, _MAT, _MAT, _MAT, _MAT, _int, _i64, _i64, _i64, _MAT, _int, _MAT, _int,
         _vp, _sz, _vp)

EXPORTED_DENSE = ("dsmoe_layer_norm", "dsmoe_layer_norm_backward_workspace_bytes", "dsmoe_layer_norm_backward",
                  "dsmoe_linear_workspace_bytes", "dsmoe_linear", "dsmoe_linear_backward_workspace_bytes",
                  "dsmoe_linear_backward", "dsmoe_gated_linear_workspace_bytes", "dsmoe_gated_linear",
                  "dsmoe_gated_linear_backward_workspace_bytes", "dsmoe_gated_linear_backward")


def _check(status: int, call: str):
    if status != 0:
        raise DsmoeError(status, call)


def _mat(t, shape, dtype, name, device=None):
    """(pointer, row stride) of a 2-D matrix with contiguous columns; (None,
    0) for None.  shape, dtype and device may be None: any."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {[rows, cols]}")
    ld, cs = t.stride()
    if cols > 1 and cs != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), ld


def _vec(t, n, name, device, dtype=None):
    """(pointer, dtype code) of a contiguous vector of n values; (None, 0)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    code = _dtype_code(t.dtype)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} values")
    return t.data_ptr(), code


def _begin(x, name):
    """The device of x (the current one) and its current stream.  The raw
    stream handle is asked for directly: a torch.cuda.Stream object takes 2.7
    us to make, as long as the launch itself."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    device = x.device
    index = device.index
    if index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {device}, but the current device is cuda:{torch.cuda.current_device()}")
    return device, torch._C._cuda_getCurrentRawStream(index)


def _new(rows, cols, dtype, device):
    """(tensor, pointer, row stride) of a new matrix."""
    t = torch.empty((rows, cols), dtype=dtype, device=device)
    return t, t.data_ptr(), cols


def _out(t, rows, cols, dtype, name, device, like=None):
    """(tensor, pointer, row stride) of an output, allocated if it is None:
    like `like`, of this shape and type, where that has no gaps (1.2 us
    instead of 1.7)."""
    if t is None:
        if like is not None and like.is_contiguous():
            t = torch.empty_like(like)
            return t, t.data_ptr(), cols
        return _new(rows, cols, dtype, device)
    p, ld = _mat(t, (rows, cols), None, name, device)
    return t, p, ld


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {tuple(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _grad_act(act, dz_dtype):
    """The act code of a backward call."""
    if dz_dtype not in (None, torch.bfloat16):
        raise TypeError("dz_dtype must be None or torch.bfloat16")
    return _act(act) | (0 if dz_dtype is None else _DZ_BF16)


def _scratch(workspace, need, device):
    """(tensor to keep alive, pointer, bytes) of the workspace of a call."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    elif workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-5, residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               total: Optional[torch.Tensor] = None):
    """Layer norm over the columns of x + residual (dsmoe_layer_norm).
    x, residual [rows][cols] bf16 or f32 (one type); gamma, beta [cols] bf16
    or f32 (one type).  y may be x or residual, and so may total.  Returns
    (y, mean f32 [rows], rstd f32 [rows], x + residual or None without a
    residual)."""
    device, stream = _begin(x, "x")
    xt = _dtype_code(x.dtype)
    xp, ldx = _mat(x, None, None, "x")
    rows, cols = x.shape
    rp, ldr = _mat(residual, (rows, cols), x.dtype, "residual", device)
    gp, gt = _vec(gamma, cols, "gamma", device)
    bp, pt = _vec(beta, cols, "beta", device, None if gamma is None else gamma.dtype)
    y, yp, ldy = _out(y, rows, cols, x.dtype, "y", device, x)
    sp, lds = None, 0
    if total is not None or residual is not None:
        total, sp, lds = _out(total, rows, cols, x.dtype, "total", device, x)
    if y.dtype != x.dtype or (total is not None and total.dtype != x.dtype):
        raise TypeError(f"y and total must be {x.dtype}")
    stats, mp, _ = _new(2, rows, torch.float32, device)
    mean, rstd = stats.unbind(0)
    _check(lib.dsmoe_layer_norm(xp, ldx, rp, ldr, xt, gp, bp, pt if gp is None else gt, rows, cols, eps, yp, ldy, sp,
                                lds, mp, mp + 4 * rows, stream), "dsmoe_layer_norm")
    return y, mean, rstd, total


def layer_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib.dsmoe_layer_norm_backward_workspace_bytes(rows, cols))


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gamma: Optional[torch.Tensor] = None, dsum: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, need_dparams: bool = True,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients of layer_norm (dsmoe_layer_norm_backward).  x is what was
    normalised (x + residual of the forward); dsum the gradient reaching it
    along the residual path.  Returns (dx, dgamma f32 [cols], dbeta f32
    [cols]), the last two None unless need_dparams."""
    device, stream = _begin(dy, "dy")
    xt = _dtype_code(dy.dtype)
    dyp, lddy = _mat(dy, None, None, "dy")
    rows, cols = dy.shape
    xp, ldx = _mat(x, (rows, cols), dy.dtype, "x", device)
    sp, lds = _mat(dsum, (rows, cols), dy.dtype, "dsum", device)
    mp, _ = _vec(mean, rows, "mean", device, torch.float32)
    rp, _ = _vec(rstd, rows, "rstd", device, torch.float32)
    gp, gt = _vec(gamma, cols, "gamma", device)
    dx, dxp, lddx = _out(dx, rows, cols, dy.dtype, "dx", device, dy)
    if dx.dtype != dy.dtype:
        raise TypeError(f"dx must be {dy.dtype}")
    dgamma = dbeta = dgp = dbp = None
    keep, wp, wn = None, None, 0
    if need_dparams:
        params, dgp, _ = _new(2, cols, torch.float32, device)
        dgamma, dbeta = params.unbind(0)
        dbp = dgp + 4 * cols
        need = lib.dsmoe_layer_norm_backward_workspace_bytes(rows, cols) if workspace is None else 0
        keep, wp, wn = _scratch(workspace, need, device)
    _check(lib.dsmoe_layer_norm_backward(dyp, lddy, xp, ldx, sp, lds, xt, gp, gt, mp, rp, rows, cols, dxp, lddx, dgp,
                                         dbp, wp, wn, stream), "dsmoe_layer_norm_backward")
    return dx, dgamma, dbeta


def linear_workspace_bytes(x: torch.Tensor, w: torch.Tensor) -> int:
    """Workspace of linear on these operands (their sizes and alignment)."""
    (xp, ldx), (wp, ldw) = _mat(x, None, torch.bfloat16, "x"), _mat(w, None, torch.bfloat16, "w")
    return int(lib.dsmoe_linear_workspace_bytes(xp, ldx, wp, ldw, x.shape[0], w.shape[0], w.shape[1]))


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, save_z: bool = False,
           y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """y = act(x W^T + bias) + residual (dsmoe_linear).  x bf16 [M][K], w bf16
    [N][K], bias bf16 or f32 [N], residual [M][N] of y's type (bf16 or f32);
    y may be residual.  Returns (y, z): z = x W^T + bias in y's type with
    save_z, else None."""
    device, stream = _begin(x, "x")
    code = _act(act)
    xp, ldx = _mat(x, None, torch.bfloat16, "x")
    wp, ldw = _mat(w, None, torch.bfloat16, "w", device)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("x and w must have the same K")
    bp, bt = _vec(bias, N, "bias", device)
    y, yp, ldy = _out(y, M, N, out_dtype, "y", device)
    yt = _dtype_code(y.dtype)
    rp, ldr = _mat(residual, (M, N), y.dtype, "residual", device)
    z, zp, ldz = _new(M, N, y.dtype, device) if save_z else (None, None, 0)
    need = lib.dsmoe_linear_workspace_bytes(xp, ldx, wp, ldw, M, N, K) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_linear(xp, ldx, wp, ldw, bp, bt, rp, ldr, code, M, N, K, yp, ldy, yt, zp, ldz, sp, sn, stream),
           "dsmoe_linear")
    return y, z


def linear_backward_workspace_bytes(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, act: str = "none",
                                    dz_dtype: Optional[torch.dtype] = None) -> int:
    """Workspace of linear_backward on these operands (their sizes and alignment)."""
    (dp, ldd), (xp, ldx), (wp, ldw) = (_mat(dy, None, torch.bfloat16, "dy"), _mat(x, None, torch.bfloat16, "x"),
                                       _mat(w, None, torch.bfloat16, "w"))
    return int(lib.dsmoe_linear_backward_workspace_bytes(dp, ldd, xp, ldx, wp, ldw, _grad_act(act, dz_dtype),
                                                         dy.shape[0], dy.shape[1], w.shape[1]))


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, z: Optional[torch.Tensor] = None,
                    act: str = "none", dx_dtype=torch.bfloat16, dw_dtype=torch.float32, need_dx: bool = True,
                    need_dw: bool = True, need_dbias: bool = False, dx: Optional[torch.Tensor] = None,
                    dw: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    dz_dtype: Optional[torch.dtype] = None):
    """Gradients of linear (dsmoe_linear_backward).  dy bf16 [M][N]; x, w the
    forward's; z the saved pre-activation (bf16 or f32), needed unless act is
    "none".  The residual's gradient is dy.  With an activation, float32
    gradients keep 16 bits of dz = dy act'(z) at twice a product's time;
    dz_dtype torch.bfloat16 rounds it to bf16 for them too, as for bf16
    gradients.  Returns (dx [M][K], dw [N][K], dbias f32 [N]), None where not
    wanted."""
    device, stream = _begin(dy, "dy")
    code = _grad_act(act, dz_dtype)
    dyp, lddy = _mat(dy, None, torch.bfloat16, "dy")
    M, N = dy.shape
    wp, ldw = _mat(w, None, torch.bfloat16, "w", device)
    K = w.shape[1]
    if w.shape[0] != N:
        raise ValueError("dy and w must have the same N")
    xp, ldx = _mat(x, (M, K), torch.bfloat16, "x", device)
    zp, ldz = _mat(z, (M, N), None, "z", device)
    zt = BF16 if z is None else _dtype_code(z.dtype)
    if act != "none" and z is None:
        raise ValueError(f"act {act!r} needs the saved z")
    dxp, lddx, dxt, dwp, lddw, dwt = None, 0, BF16, None, 0, F32
    if dx is not None or need_dx:
        dx, dxp, lddx = _out(dx, M, K, dx_dtype, "dx", device)
        dxt = _dtype_code(dx.dtype)
    if dw is not None or need_dw:
        dw, dwp, lddw = _out(dw, N, K, dw_dtype, "dw", device)
        dwt = _dtype_code(dw.dtype)
    dbias = torch.empty((N,), dtype=torch.float32, device=device) if need_dbias else None
    need = lib.dsmoe_linear_backward_workspace_bytes(dyp, lddy, xp, ldx, wp, ldw, code, M, N, K) \
        if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_linear_backward(dyp, lddy, xp, ldx, wp, ldw, zp, ldz, zt, code, M, N, K, dxp, lddx,
                                     dxt, dwp, lddw, dwt, None if dbias is None else dbias.data_ptr(), sp, sn, stream),
           "dsmoe_linear_backward")
    return dx, dw, dbias


def gated_linear_workspace_bytes(x: torch.Tensor, w13: torch.Tensor) -> int:
    """Workspace of gated_linear on these operands (their sizes and alignment)."""
    (xp, ldx), (wp, ldw) = _mat(x, None, torch.bfloat16, "x"), _mat(w13, None, torch.bfloat16, "w13")
    return int(lib.dsmoe_gated_linear_workspace_bytes(xp, ldx, wp, ldw, x.shape[0], w13.shape[1],
                                                      w13.shape[0] // 2))


def gated_linear(x: torch.Tensor, w13: torch.Tensor, act: str = "silu", out_dtype=torch.bfloat16,
                 save_h: bool = False, a: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """a = act(x Wg^T) * (x Wu^T) with w13 = [Wg; Wu] (dsmoe_gated_linear).
    x bf16 [M][H], w13 bf16 [2I][H], gate rows first.  Returns (a [M][I], h):
    h = x w13^T bf16 [M][2I] with save_h, else None."""
    device, stream = _begin(x, "x")
    code = _act(act)
    xp, ldx = _mat(x, None, torch.bfloat16, "x")
    wp, ldw = _mat(w13, None, torch.bfloat16, "w13", device)
    M, H = x.shape
    I = w13.shape[0] // 2
    if w13.shape[1] != H or w13.shape[0] != 2 * I:
        raise ValueError("w13 must be [2I][H] with x's H")
    a, ap, lda = _out(a, M, I, out_dtype, "a", device)
    at = _dtype_code(a.dtype)
    h, hp, ldh = _new(M, 2 * I, torch.bfloat16, device) if save_h else (None, None, 0)
    need = lib.dsmoe_gated_linear_workspace_bytes(xp, ldx, wp, ldw, M, H, I) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_gated_linear(xp, ldx, wp, ldw, code, M, H, I, ap, lda, at, hp, ldh, sp, sn, stream),
           "dsmoe_gated_linear")
    return a, h


def gated_linear_backward_workspace_bytes(x: torch.Tensor, w13: torch.Tensor) -> int:
    """Workspace of gated_linear_backward on these operands (their sizes and alignment)."""
    (xp, ldx), (wp, ldw) = _mat(x, None, torch.bfloat16, "x"), _mat(w13, None, torch.bfloat16, "w13")
    return int(lib.dsmoe_gated_linear_backward_workspace_bytes(xp, ldx, wp, ldw, x.shape[0], w13.shape[1],
                                                               w13.shape[0] // 2))


def gated_linear_backward(da: torch.Tensor, x: torch.Tensor, w13: torch.Tensor, h: torch.Tensor, act: str = "silu",
                          dx_dtype=torch.bfloat16, dw_dtype=torch.float32, need_dx: bool = True,
                          need_dw: bool = True, dx: Optional[torch.Tensor] = None,
                          dw13: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          dz_dtype: Optional[torch.dtype] = None):
    """Gradients of gated_linear (dsmoe_gated_linear_backward) from the saved
    h.  da bf16 [M][I].  Float32 gradients keep 16 bits of the gradient at h, at
    twice a product's time; dz_dtype as in linear_backward.  Returns (dx
    [M][H], dw13 [2I][H]), None where not wanted."""
    device, stream = _begin(da, "da")
    code = _grad_act(act, dz_dtype)
    dap, ldda = _mat(da, None, torch.bfloat16, "da")
    M, I = da.shape
    wp, ldw = _mat(w13, None, torch.bfloat16, "w13", device)
    H = w13.shape[1]
    if w13.shape[0] != 2 * I:
        raise ValueError("w13 must be [2I][H] with da's I")
    xp, ldx = _mat(x, (M, H), torch.bfloat16, "x", device)
    hp, ldh = _mat(h, (M, 2 * I), torch.bfloat16, "h", device)
    dxp, lddx, dxt, dwp, lddw, dwt = None, 0, BF16, None, 0, F32
    if dx is not None or need_dx:
        dx, dxp, lddx = _out(dx, M, H, dx_dtype, "dx", device)
        dxt = _dtype_code(dx.dtype)
    if dw13 is not None or need_dw:
        dw13, dwp, lddw = _out(dw13, 2 * I, H, dw_dtype, "dw13", device)
        dwt = _dtype_code(dw13.dtype)
    need = lib.dsmoe_gated_linear_backward_workspace_bytes(xp, ldx, wp, ldw, M, H, I) if workspace is None else 0
    keep, sp, sn = _scratch(workspace, need, device)
    _check(lib.dsmoe_gated_linear_backward(dap, ldda, xp, ldx, wp, ldw, hp, ldh, code, M, H, I, dxp, lddx,
                                           dxt, dwp, lddw, dwt, sp, sn, stream),
           "dsmoe_gated_linear_backward")
    return dx, dw13


def dense_ffn_forward(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                      w13: torch.Tensor, w2: torch.Tensor, residual: Optional[torch.Tensor] = None, act: str = "silu",
                      eps: float = 1e-5, training: bool = False):
    """The dense feed-forward sub-layer of a pre-norm block:

        s = x + residual,  y = s + gated_linear(layer_norm(s), w13) w2^T

    x, residual bf16 [T][H], w13 bf16 [2I][H], w2 bf16 [H][I].  Returns (y,
    saved): y bf16 [T][H] and, when training, what dense_ffn_backward needs."""
    n, mean, rstd, s = layer_norm(x, gamma, beta, eps, residual)
    if s is None:
        s = x
    a, h = gated_linear(n, w13, act, save_h=training)
    y, _ = linear(a, w2, residual=s)
    return y, ({"s": s, "mean": mean, "rstd": rstd, "n": n, "h": h, "a": a} if training else None)


def dense_ffn_backward(dy: torch.Tensor, saved: dict, gamma: Optional[torch.Tensor], w13: torch.Tensor,
                       w2: torch.Tensor, act: str = "silu", dw_dtype=torch.float32,
                       dz_dtype: Optional[torch.dtype] = None):
    """Gradients of dense_ffn_forward from dy bf16 [T][H] and its saved dict;
    dz_dtype as in gated_linear_backward.  Returns {"dx" (of x and of residual
    alike), "dgamma", "dbeta", "dw13", "dw2"}."""
    da, dw2, _ = linear_backward(dy, saved["a"], w2, dw_dtype=dw_dtype)
    dn, dw13 = gated_linear_backward(da, saved["n"], w13, saved["h"], act, dw_dtype=dw_dtype, dz_dtype=dz_dtype)
    dx, dgamma, dbeta = layer_norm_backward(dn, saved["s"], saved["mean"], saved["rstd"], gamma, dsum=dy)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta, "dw13": dw13, "dw2": dw2}
