"""Host-side checks of the dense feed-forward calls (no GPU needed): exports,
the C header, workspace sizes, and the refusal of invalid arguments before any
device is touched."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 1)
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 5


@pytest.fixture
def d():
    import fp8_block_scaled_dsmoe_amd as d
    return d


def test_library_exports_every_declared_function(d):
    src = open(os.path.join(ROOT, "include", "dsmoe_dense.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(dsmoe_[a-z0-9_]+)\s*\(", src)))
    assert sorted(d.EXPORTED_DENSE) == names
    for n in names:
        assert hasattr(d.lib, n), n


def _call(f, defaults, **change):
    args = dict(defaults)
    assert not set(change) - set(args), set(change) - set(args)
    args.update(change)
    return f(*args.values())


def _norm(d, **c):
    return _call(d.lib.dsmoe_layer_norm, dict(
        x=A, ldx=64, residual=None, ldr=0, xt=0, gamma=A, beta=A, pt=0, rows=4, cols=64, eps=1e-5, y=A, ldy=64,
        sum=None, lds=0, mean=A, rstd=A, stream=None), **c)


def test_layer_norm_refusals(d):
    assert _norm(d, xt=2) == DTYPE and _norm(d, pt=-1) == DTYPE
    assert _norm(d, rows=-1) == SHAPE and _norm(d, rows=1 << 31) == SHAPE
    assert _norm(d, cols=0) == SHAPE and _norm(d, cols=4194305) == SHAPE
    assert _norm(d, ldx=63) == SHAPE and _norm(d, ldy=63) == SHAPE and _norm(d, ldx=4194305) == SHAPE
    assert _norm(d, residual=A, ldr=63) == SHAPE and _norm(d, sum=A, lds=0) == SHAPE
    assert _norm(d, eps=-1.0) == SHAPE and _norm(d, eps=float("nan")) == SHAPE and _norm(d, eps=float("inf")) == SHAPE
    assert _norm(d, x=None) == NULL and _norm(d, y=None) == NULL
    assert _norm(d, x=ODD) == ALIGN and _norm(d, gamma=ODD) == ALIGN and _norm(d, mean=ODD) == ALIGN
    assert _norm(d, x=None, y=None, rows=0) == OK


def _norm_bwd(d, **c):
    return _call(d.lib.dsmoe_layer_norm_backward, dict(
        dy=A, lddy=64, x=A, ldx=64, dsum=None, ldds=0, xt=0, gamma=A, pt=0, mean=A, rstd=A, rows=4, cols=64, dx=A,
        lddx=64, dgamma=A, dbeta=A, ws=A, wsn=1 << 30, stream=None), **c)


def test_layer_norm_backward_refusals(d):
    assert _norm_bwd(d, xt=3) == DTYPE
    assert _norm_bwd(d, cols=0) == SHAPE and _norm_bwd(d, lddx=1) == SHAPE and _norm_bwd(d, dsum=A, ldds=1) == SHAPE
    for name in ("dy", "x", "mean", "rstd", "dx", "dgamma", "dbeta"):
        assert _norm_bwd(d, **{name: None}) == NULL, name
    for name in ("dy", "x", "mean", "rstd", "dx", "dgamma", "dbeta", "gamma"):
        assert _norm_bwd(d, **{name: ODD}) == ALIGN, name
    need = d.layer_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert _norm_bwd(d, wsn=need - 1) == WORKSPACE and _norm_bwd(d, ws=None) == WORKSPACE
    assert _norm_bwd(d, ws=ctypes.c_void_p((1 << 20) + 64)) == ALIGN
    assert _norm_bwd(d, rows=0, dgamma=None, dbeta=None) == OK


def _linear(d, **c):
    return _call(d.lib.dsmoe_linear, dict(
        x=A, ldx=64, w=A, ldw=64, bias=None, bt=0, residual=None, ldr=0, act=0, M=4, N=32, K=64, y=A, ldy=32, yt=0,
        z=None, ldz=0, ws=None, wsn=0, stream=None), **c)


def test_linear_refusals(d):
    assert _linear(d, yt=5) == DTYPE and _linear(d, bt=5) == DTYPE
    assert _linear(d, act=4) == SHAPE and _linear(d, act=-1) == SHAPE
    for name in ("N", "K"):
        assert _linear(d, **{name: 0}) == SHAPE and _linear(d, **{name: 4194305}) == SHAPE
    assert _linear(d, M=-1) == SHAPE
    assert _linear(d, ldx=63) == SHAPE and _linear(d, ldw=63) == SHAPE and _linear(d, ldy=31) == SHAPE
    assert _linear(d, z=A, ldz=31) == SHAPE and _linear(d, residual=A, ldr=31) == SHAPE
    for name in ("x", "w", "y"):
        assert _linear(d, **{name: None}) == NULL
        assert _linear(d, **{name: ODD}) == ALIGN
    assert _linear(d, bias=ODD) == ALIGN and _linear(d, residual=ODD, ldr=32) == ALIGN
    assert _linear(d, M=0, x=None, w=None, y=None) == OK
    # operands that are not 16-byte rows need a workspace for their copies
    x2 = ctypes.c_void_p((1 << 20) + 2)
    need = d.lib.dsmoe_linear_workspace_bytes(x2, 64, A, 64, 4, 32, 64)
    assert need >= d.lib.dsmoe_linear_workspace_bytes(A, 64, A, 64, 4, 32, 64)
    if need:
        assert _linear(d, x=x2, ws=A, wsn=need - 1) == WORKSPACE
        assert _linear(d, x=x2) == WORKSPACE


def _linear_bwd(d, **c):
    return _call(d.lib.dsmoe_linear_backward, dict(
        dy=A, lddy=32, x=A, ldx=64, w=A, ldw=64, z=A, ldz=32, zt=0, act=1, M=4, N=32, K=64, dx=A, lddx=64, dxt=0,
        dw=A, lddw=64, dwt=1, dbias=A, ws=A, wsn=1 << 30, stream=None), **c)


def test_linear_backward_refusals(d):
    assert _linear_bwd(d, zt=9) == DTYPE and _linear_bwd(d, dxt=9) == DTYPE and _linear_bwd(d, dwt=9) == DTYPE
    assert _linear_bwd(d, act=9) == SHAPE and _linear_bwd(d, N=0) == SHAPE and _linear_bwd(d, lddy=31) == SHAPE
    assert _linear_bwd(d, lddw=63) == SHAPE and _linear_bwd(d, lddx=63) == SHAPE and _linear_bwd(d, ldz=31) == SHAPE
    for name in ("dy", "x", "w", "z"):
        assert _linear_bwd(d, **{name: None}) == NULL, name
        assert _linear_bwd(d, **{name: ODD}) == ALIGN, name
    for name in ("dx", "dw", "dbias"):
        assert _linear_bwd(d, **{name: ODD}) == ALIGN, name
    need = d.lib.dsmoe_linear_backward_workspace_bytes(A, 32, A, 64, A, 64, 1, 4, 32, 64)
    assert need > 0
    assert _linear_bwd(d, wsn=need - 1) == WORKSPACE and _linear_bwd(d, ws=None) == WORKSPACE
    assert _linear_bwd(d, dx=None, dw=None, dbias=None) == OK
    assert _linear_bwd(d, M=0, dw=None, dbias=None) == OK


def _gated(d, **c):
    return _call(d.lib.dsmoe_gated_linear, dict(
        x=A, ldx=64, w13=A, ldw=64, act=1, M=4, H=64, I=32, a=A, lda=32, at=0, h=None, ldh=0, ws=None, wsn=0,
        stream=None), **c)


def test_gated_linear_refusals(d):
    assert _gated(d, at=2) == DTYPE
    assert _gated(d, act=7) == SHAPE and _gated(d, I=0) == SHAPE and _gated(d, I=2097153) == SHAPE
    assert _gated(d, I=1 << 62) == SHAPE and _gated(d, H=0) == SHAPE
    assert _gated(d, lda=31) == SHAPE and _gated(d, h=A, ldh=63) == SHAPE and _gated(d, ldw=63) == SHAPE
    for name in ("x", "w13", "a"):
        assert _gated(d, **{name: None}) == NULL and _gated(d, **{name: ODD}) == ALIGN
    assert _gated(d, h=ODD, ldh=64) == ALIGN
    assert _gated(d, M=0, x=None) == OK


def _gated_bwd(d, **c):
    return _call(d.lib.dsmoe_gated_linear_backward, dict(
        da=A, ldda=32, x=A, ldx=64, w13=A, ldw=64, h=A, ldh=64, act=1, M=4, H=64, I=32, dx=A, lddx=64, dxt=0, dw=A,
        lddw=64, dwt=1, ws=A, wsn=1 << 30, stream=None), **c)


def test_gated_linear_backward_refusals(d):
    assert _gated_bwd(d, dxt=2) == DTYPE and _gated_bwd(d, dwt=2) == DTYPE
    assert _gated_bwd(d, act=-2) == SHAPE and _gated_bwd(d, ldh=63) == SHAPE and _gated_bwd(d, lddw=63) == SHAPE
    for name in ("da", "x", "w13", "h"):
        assert _gated_bwd(d, **{name: None}) == NULL and _gated_bwd(d, **{name: ODD}) == ALIGN
    need = d.lib.dsmoe_gated_linear_backward_workspace_bytes(A, 64, A, 64, 4, 64, 32)
    assert need >= 4 * 64 * 2
    assert _gated_bwd(d, wsn=need - 1) == WORKSPACE and _gated_bwd(d, ws=None) == WORKSPACE
    assert _gated_bwd(d, dx=None, dw=None) == OK
    assert _gated_bwd(d, M=0, dw=None) == OK


def test_forward_workspace_refusals(d):
    """Sizes that split K or copy an operand, so that a workspace is needed."""
    ws = ctypes.c_void_p(1 << 21)
    for call, query, size in (
            (_linear, d.lib.dsmoe_linear_workspace_bytes, dict(M=769, N=264, K=3856)),
            (_gated, d.lib.dsmoe_gated_linear_workspace_bytes, dict(M=328, H=3880, I=328))):
        M, a, b = size.values()
        K, N = (b, a) if "K" in size else (a, b)
        wide = dict(ldx=K, ldw=K, **({"ldy": N} if "K" in size else {"lda": N}), **size)
        aligned, packed = query(A, K, A, K, *size.values()), query(ctypes.c_void_p((1 << 20) + 2), K, A, K, *size.values())
        assert aligned > 0 and packed >= aligned + M * K * 2
        for need, x in ((aligned, A), (packed, ctypes.c_void_p((1 << 20) + 2))):
            assert call(d, **wide, x=x, ws=ws, wsn=need - 1) == WORKSPACE
            assert call(d, **wide, x=x, ws=None, wsn=need) == WORKSPACE
            assert call(d, **wide, x=x) == WORKSPACE
            assert call(d, **wide, x=x, ws=ctypes.c_void_p((1 << 21) + 128), wsn=need) == ALIGN


def test_backward_calls_take_the_bf16_dz_flag_and_no_other(d):
    flag = 16
    args = (A, 32, A, 64, A, 64)
    size = d.lib.dsmoe_linear_backward_workspace_bytes
    # dz of an activation keeps the rest of its rounding unless told not to
    assert size(*args, 1, 128, 32, 64) - size(*args, 1 | flag, 128, 32, 64) == 128 * 32 * 2
    assert size(*args, 0, 128, 32, 64) == size(*args, flag, 128, 32, 64)
    for call in (_linear_bwd, _gated_bwd):
        assert call(d, act=3 | flag, ws=None) == WORKSPACE
        assert call(d, act=4 | flag) == SHAPE and call(d, act=2 * flag) == SHAPE and call(d, act=3 * flag) == SHAPE
    assert _linear(d, act=1 | flag) == SHAPE and _gated(d, act=1 | flag) == SHAPE
    need = size(*args, 1 | flag, 4, 32, 64)
    assert _linear_bwd(d, act=1 | flag, wsn=need - 1) == WORKSPACE


def test_python_refusals(d):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        d.layer_norm(x)                       # a host tensor
    with pytest.raises(ValueError):
        d.linear(x, x)
    with pytest.raises(TypeError):
        d.gated_linear([1.0], x)


C_PROGRAM = r"""
#include <stdio.h>
#include "dsmoe_dense.h"
int main(void) {
  if (dsmoe_layer_norm_backward_workspace_bytes(0, 0) != 0) return 1;
  if (dsmoe_linear(NULL, 0, NULL, 0, NULL, DSMOE_BF16, NULL, 0, DSMOE_ACT_GELU, 4, 0, 8, NULL, 0, DSMOE_F32, NULL, 0,
                   NULL, 0, NULL) != DSMOE_ERR_SHAPE) return 2;
  puts("ok");
  return 0;
}
"""


def test_header_is_c99_and_links_from_c(tmp_path, d):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "dense.c", tmp_path / "dense"
    src.write_text(C_PROGRAM)
    libdir = os.path.dirname(d.LIB_PATH)
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-L", libdir, "-ldsmoe",
                        f"-Wl,-rpath,{libdir}", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", (out.returncode, out.stderr)


def test_sizes_that_run_every_dense_kernel(d):
    """Each size of dense_kernels.SIZES takes the kernels that its GPU test is
    there for, and together they are every tile shape in every form."""
    import dense_kernels as dk
    for size, want in dk.SIZES.items():
        assert dk.kernels(d.lib, *size) == want, size
    for product in dk.PRODUCTS:
        rows = [v for k, v in dk.SIZES.items() if k[0] == product]
        assert {s for s, split, rest in rows if not split and not rest} == set(dk.SHAPES), product
        assert {rest for _, _, rest in rows if rest} == set(dk.SHAPES) - {"256x256"}, product
        assert any(split for _, split, _ in rows), product
    # what gated backward runs on a training batch: both products cut in two
    for product in ("dx", "dw"):
        assert dk.kernels(d.lib, product, 4096, 2 * 2048, 7168) == ("256x256", False, "256x192")
    assert dk.kernels(d.lib, "y", 4, 32, 64)[0] == dk.kernels(d.lib, "gated", 64, 64, 64)[0] == "few tokens"
    f = d.lib.dsmoe_dense_kernels
    out = (ctypes.c_int64 * 6)()
    for bad in ((4, 8, 8, 8), (-1, 8, 8, 8), (0, 0, 8, 8), (0, 8, 0, 8), (0, 8, 8, 0), (0, (1 << 28) + 1, 8, 8)):
        assert f(*bad, ctypes.byref(out)) == SHAPE
