"""Host-side checks of the experts' calls outside FP8 (no GPU needed): exports, the
C header, workspace sizes, and the refusal of invalid arguments before any
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
    src = open(os.path.join(ROOT, "include", "dsmoe_experts.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(dsmoe_[a-z0-9_]+)\s*\(", src)))
    assert sorted(d.EXPORTED_EXPERTS) == names
    for n in names:
        assert hasattr(d.lib, n), n


def _call(f, defaults, **change):
    args = dict(defaults)
    assert not set(change) - set(args), set(change) - set(args)
    args.update(change)
    return f(*args.values())


def _linear(d, **c):
    return _call(d.lib.dsmoe_grouped_linear, dict(
        x=A, ldx=64, n=4, rows=None, w=A, ldw=64, offsets=A, G=2, R=4, N=32, K=64, y=A, ldy=32, yt=0, ws=None, wsn=0,
        stream=None), **c)


def _gated(d, **c):
    return _call(d.lib.dsmoe_grouped_gated_linear, dict(
        x=A, ldx=64, n=4, rows=None, w=A, ldw=64, scale=A, act=1, offsets=A, G=2, R=4, H=64, I=32, y=A, ldy=32, yt=0,
        h=None, ldh=0, ws=None, wsn=0, stream=None), **c)


def _int8(d, **c):
    return _call(d.lib.dsmoe_int8_linear, dict(
        x=A, ldx=64, xs=A, n=4, rows=None, w=A, ldw=64, ws_=A, offsets=A, G=2, R=4, N=32, K=64, y=A, ldy=32, yt=0,
        ws=None, wsn=0, stream=None), **c)


def _int8_gated(d, **c):
    return _call(d.lib.dsmoe_int8_gated_linear, dict(
        x=A, ldx=64, xs=A, n=4, rows=None, w=A, ldw=64, ws_=A, scale=None, act=1, offsets=A, G=2, R=4, H=64, I=32, y=A,
        ldy=32, yt=0, ws=None, wsn=0, stream=None), **c)


def test_forward_refusals(d):
    for f, n, k in ((_linear, "N", "K"), (_gated, "I", "H"), (_int8, "N", "K"), (_int8_gated, "I", "H")):
        assert f(d, yt=2) == DTYPE and f(d, yt=-1) == DTYPE
        assert f(d, G=0) == SHAPE and f(d, G=1025) == SHAPE and f(d, offsets=None) == SHAPE
        assert f(d, R=-1) == SHAPE and f(d, R=1 << 31) == SHAPE and f(d, R=5) == SHAPE    # R is n without an index
        assert f(d, n=-1, rows=A) == SHAPE and f(d, n=0, rows=A) == SHAPE and f(d, n=1 << 31, rows=A) == SHAPE
        for v in (n, k):
            assert f(d, **{v: 0}) == SHAPE and f(d, **{v: 4194305}) == SHAPE
        assert f(d, ldx=63) == SHAPE and f(d, ldw=63) == SHAPE and f(d, ldy=31) == SHAPE and f(d, ldx=4194305) == SHAPE
        for v in ("x", "w", "y"):
            assert f(d, **{v: None}) == NULL, v
        assert f(d, y=ODD) == ALIGN and f(d, rows=ODD) == ALIGN and f(d, offsets=ODD) == ALIGN
        assert f(d, R=0, n=0, x=None, w=None, y=None) == OK
        assert f(d, R=0, n=9, rows=A, x=None, w=None, y=None) == OK
    for f in (_linear, _gated):
        assert f(d, x=ODD) == ALIGN and f(d, w=ODD) == ALIGN
    for f in (_gated, _int8_gated):
        assert f(d, act=4) == SHAPE and f(d, act=-1) == SHAPE and f(d, act=17) == SHAPE and f(d, scale=ODD) == ALIGN
        assert f(d, I=2097153) == SHAPE
    assert _gated(d, h=A, ldh=63) == SHAPE and _gated(d, h=ODD, ldh=64) == ALIGN
    for f, k in ((_int8, "K"), (_int8_gated, "H")):
        assert f(d, xs=None) == NULL and f(d, ws_=None) == NULL and f(d, xs=ODD) == ALIGN and f(d, ws_=ODD) == ALIGN
        assert f(d, ldx=131072, ldw=131072, **{k: 131072}) == SHAPE


def _linear_bwd(d, **c):
    return _call(d.lib.dsmoe_grouped_linear_backward, dict(
        dy=A, lddy=32, n_dy=4, dy_rows=None, x=A, ldx=64, n=4, rows=None, w=A, ldw=64, offsets=A, G=2, R=4, N=32, K=64,
        dx=A, lddx=64, dxt=0, dw=A, lddw=64, dwt=1, ws=None, wsn=0, stream=None), **c)


def _gated_bwd(d, **c):
    return _call(d.lib.dsmoe_grouped_gated_linear_backward, dict(
        da=A, ldda=32, x=A, ldx=64, n=4, rows=None, w=A, ldw=64, h=A, ldh=64, scale=A, act=1, offsets=A, G=2, R=4, H=64,
        I=32, dx=A, lddx=64, dxt=0, dw=A, lddw=64, dwt=1, ds=A, ws=A, wsn=1 << 30, stream=None), **c)


def test_backward_refusals(d):
    for f in (_linear_bwd, _gated_bwd):
        assert f(d, dxt=2) == DTYPE and f(d, dwt=9) == DTYPE
        assert f(d, G=0) == SHAPE and f(d, G=1025) == SHAPE and f(d, offsets=None) == SHAPE and f(d, R=5) == SHAPE
        assert f(d, n=0, rows=A) == SHAPE and f(d, ldx=63) == SHAPE and f(d, lddx=63) == SHAPE and f(d, lddw=63) == SHAPE
        for v in ("x", "w", "dx", "dw", "rows", "offsets"):
            assert f(d, **{v: ODD}) == ALIGN, v
        assert f(d, x=None) == NULL and f(d, w=None) == NULL
        assert f(d, dx=None, dw=None, **({"ds": None} if f is _gated_bwd else {})) == OK
        assert f(d, R=0, n=0, dw=None, **({} if f is _gated_bwd else {"n_dy": 0})) == OK
    assert _linear_bwd(d, dy=None) == NULL and _linear_bwd(d, dy=ODD) == ALIGN and _linear_bwd(d, lddy=31) == SHAPE
    assert _linear_bwd(d, n_dy=5) == SHAPE and _linear_bwd(d, n_dy=0, dy_rows=A) == SHAPE
    assert _linear_bwd(d, dy_rows=ODD) == ALIGN
    assert _gated_bwd(d, da=None) == NULL and _gated_bwd(d, h=None) == NULL and _gated_bwd(d, da=ODD) == ALIGN
    assert _gated_bwd(d, h=ODD) == ALIGN and _gated_bwd(d, ldh=63) == SHAPE and _gated_bwd(d, ldda=31) == SHAPE
    assert _gated_bwd(d, scale=ODD) == ALIGN and _gated_bwd(d, ds=ODD) == ALIGN
    for act in (4, -1, 32, 20, 48):
        assert _gated_bwd(d, act=act) == SHAPE, act


def test_workspace_refusals(d):
    """Operands that need copies: a pointer off 16 bytes, a row length off whole
    16 bytes, rows by index in a weight gradient."""
    off2 = ctypes.c_void_p((1 << 20) + 2)
    size = d.lib.dsmoe_grouped_linear_workspace_bytes
    need = size(off2, 64, 4, None, A, 64, 2, 4, 32, 64)
    assert need == 512 and size(A, 64, 4, None, A, 64, 2, 4, 32, 64) == 0
    for ws, n in ((A, need - 1), (None, need), (None, 0)):
        assert _linear(d, x=off2, ws=ws, wsn=n) == WORKSPACE
    assert _linear(d, x=off2, ws=ctypes.c_void_p((1 << 20) + 64), wsn=need) == ALIGN
    size = d.lib.dsmoe_grouped_linear_backward_workspace_bytes
    need = size(A, 32, 9, A, A, 64, 4, None, A, 64, 2, 4, 32, 64)
    assert need >= 4 * 32 * 2
    assert _linear_bwd(d, n_dy=9, dy_rows=A, ws=A, wsn=need - 1) == WORKSPACE
    size = d.lib.dsmoe_grouped_gated_linear_backward_workspace_bytes
    need = size(A, 64, 4, None, A, 64, 2, 4, 64, 32)
    assert need >= 4 * 64 * 2
    assert _gated_bwd(d, wsn=need - 1) == WORKSPACE and _gated_bwd(d, ws=None) == WORKSPACE
    assert _gated_bwd(d, act=3 | 16, ws=None) == WORKSPACE
    # rows by index that span 2^31 bytes or more are gathered first
    size = d.lib.dsmoe_grouped_linear_workspace_bytes
    assert size(A, 4194304, 300, A, A, 64, 2, 4, 32, 64) == 512 and size(A, 4194304, 200, A, A, 64, 2, 4, 32, 64) == 0
    # invalid sizes
    assert size(A, 64, 4, None, A, 64, 0, 4, 32, 64) == 0 and size(A, 64, 5, None, A, 64, 2, 4, 32, 64) == 0
    assert d.lib.dsmoe_int8_linear_workspace_bytes(A, 72, 4, None, A, 72, 2, 4, 32, 72) > 0


def test_router_and_quantiser_refusals(d):
    def router(**c):
        return _call(d.lib.dsmoe_router_backward, dict(dgate=A, top=A, logits=A, T=4, E=16, K=2, out=A, stream=None), **c)

    assert router(T=-1) == SHAPE and router(E=0) == SHAPE and router(E=1025) == SHAPE and router(K=0) == SHAPE
    assert router(K=33) == SHAPE and router(K=17) == SHAPE and router(T=0, dgate=None) == OK
    for v in ("dgate", "top", "logits", "out"):
        assert router(**{v: None}) == NULL and router(**{v: ODD}) == ALIGN

    def quant(**c):
        return _call(d.lib.dsmoe_quant_rows_int8, dict(x=A, ldx=64, xt=0, rows=4, cols=64, q=ODD, ldq=64, scale=A,
                                                       stream=None), **c)

    assert quant(xt=2) == DTYPE and quant(rows=-1) == SHAPE and quant(cols=0) == SHAPE and quant(ldx=63) == SHAPE
    assert quant(ldq=63) == SHAPE and quant(cols=4194305) == SHAPE
    for v in ("x", "q", "scale"):
        assert quant(**{v: None}) == NULL
    assert quant(x=ODD) == ALIGN and quant(scale=ODD) == ALIGN and quant(rows=0, x=None, q=None, scale=None) == OK


def test_python_refusals(d):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        d.grouped_linear(x, w, None)              # a host tensor
    with pytest.raises(TypeError):
        d.grouped_gated_linear([1.0], w, None)
    with pytest.raises(ValueError):
        d.quant_rows_int8(x)
    with pytest.raises(ValueError):
        d.int8_linear(x, x, w, x)
    with pytest.raises(ValueError):
        d.moe_ffn_forward(x, {}, w, w, n_shared=2)


def test_weights_of_experts_are_rows_of_one_matrix(d):
    cpu = torch.device("cpu")
    w = torch.zeros((3, 4, 8), dtype=torch.bfloat16)
    take = lambda t: d.experts._experts(t, torch.bfloat16, "w", cpu)[1:]
    assert take(w) == (8, 3, 4, 8)
    assert take(w[0]) == (8, 1, 4, 8)
    wide = torch.zeros((3, 4, 16), dtype=torch.bfloat16)[:, :, 3:11]
    assert take(wide) == (16, 3, 4, 8)
    assert take(torch.zeros((3, 1, 16), dtype=torch.bfloat16)[:, :, :8]) == (16, 3, 1, 8)
    assert take(torch.zeros((1, 1, 16), dtype=torch.bfloat16)[:, :, :8]) == (8, 1, 1, 8)
    for bad in (w[:, :2], w.transpose(0, 1), w.transpose(1, 2), w[:1].expand(3, 4, 8), w[:, :1].expand(3, 4, 8),
                w[0, :1].expand(4, 8)):
        with pytest.raises(ValueError):
            take(bad)
    with pytest.raises(TypeError):
        take(w.float())


def test_sizes_that_run_every_grouped_kernel(d):
    """Each size of grouped_kernels.SIZES takes the kernel that its GPU test is there
    for, and together they are every tile shape of every product."""
    import grouped_kernels as gk
    for size, want in gk.SIZES.items():
        assert gk.shape(d.lib, *size) == want, size
        s = gk.group_sizes(size[1], size[2])
        assert len(s) == size[1] and sum(s) == size[2] and min(s) >= 0
    for product in gk.PRODUCTS:
        shapes = {s for k, s in gk.SIZES.items() if k[0] == product}
        missing = {"32x128"} if product == "dw" else set()
        if product not in ("y", "int8"):
            missing = missing | {"256x256 each"}
        assert shapes == set(gk.SHAPES) - missing, product
    assert gk.shape(d.lib, "y", 0, 8, 8, 8) is None and gk.shape(d.lib, "y", 1, 0, 8, 8) is None
    # what sizes of the framework take
    assert gk.shape(d.lib, "gated", 256, 8, 2048, 7168) == "64x64"
    assert gk.shape(d.lib, "y", 256, 512, 7168, 2048) == "32x128"
    assert gk.shape(d.lib, "gated", 256, 32768, 2048, 7168) == "256x256"
    assert gk.shape(d.lib, "dw", 32, 16384, 4096, 7168) == "256x256"


def test_sizes_past_the_card_are_refused(d):
    """Numbers of elements past 2^40, whose tiles would not be counted in 32 bits."""
    big = dict(ldx=4194304, ldw=4194304, ldy=4194304)
    assert _linear(d, N=4194304, K=4194304, **big) == SHAPE
    assert _linear(d, N=4194304, K=64, R=(1 << 31) - 1, n=(1 << 31) - 1, **big) == SHAPE
    assert _int8(d, N=4194304, K=131071, G=1024, **big) == SHAPE
    assert _gated(d, I=2097152, H=4194304, **big) == SHAPE
    wide = dict(lddy=4194304, ldx=4194304, ldw=4194304, lddx=4194304, lddw=4194304)
    assert _linear_bwd(d, N=4194304, K=4194304, **wide) == SHAPE
    assert d.lib.dsmoe_grouped_linear_workspace_bytes(A, 4194304, 4, None, A, 4194304, 2, 4, 4194304, 4194304) == 0


def test_tokens_of_the_pass_are_the_routing_s(d):
    i32, b16 = torch.int32, torch.bfloat16
    routing = {"offsets": torch.zeros(3, dtype=i32), "perm": torch.zeros(8, dtype=i32),
               "inv": torch.zeros((4, 2), dtype=i32), "gates": torch.zeros((4, 2))}
    w13, w2 = torch.zeros((2, 16, 8), dtype=b16), torch.zeros((2, 8, 8), dtype=b16)
    x, short = torch.zeros((4, 8), dtype=b16), torch.zeros((3, 8), dtype=b16)
    with pytest.raises(ValueError, match="tokens"):
        d.moe_ffn_forward(short, routing, w13, w2)
    with pytest.raises(ValueError, match="tokens"):
        d.moe_ffn_int8_forward(short, routing, (w13, None), (w2, None))
    with pytest.raises(ValueError, match="n_shared"):
        d.moe_ffn_forward(x, routing, w13, w2, n_shared=2)
    saved = {"offsets": routing["offsets"], "perm": routing["perm"], "scale": None, "shared0": -1, "a": None, "h": None}
    for dy, y in ((short, x), (short, short)):
        with pytest.raises(ValueError, match="routing"):
            d.moe_ffn_backward(dy, y, routing, w13, w2, saved)


C_PROGRAM = r"""
#include <stdio.h>
#include "dsmoe_experts.h"
int main(void) {
  if (dsmoe_grouped_linear_workspace_bytes(NULL, 0, 0, NULL, NULL, 0, 0, 0, 0, 0) != 0) return 1;
  if (dsmoe_int8_linear(NULL, 0, NULL, 4, NULL, NULL, 0, NULL, NULL, 1, 4, 8, DSMOE_INT8_MAX_K, NULL, 0, DSMOE_F32, NULL,
                        0, NULL) != DSMOE_ERR_SHAPE) return 2;
  puts("ok");
  return 0;
}
"""


def test_header_is_c99_and_links_from_c(tmp_path, d):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "experts.c", tmp_path / "experts"
    src.write_text(C_PROGRAM)
    libdir = os.path.dirname(d.LIB_PATH)
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-L", libdir, "-ldsmoe",
                        f"-Wl,-rpath,{libdir}", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", (out.returncode, out.stderr)
