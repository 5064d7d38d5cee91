"""Sizes that together run every kernel of the grouped products (not collected: no
test_ prefix).  What a size runs is asked of the library, so a change of its rule
that takes a size elsewhere fails test_experts_abi_cpu.py."""

import ctypes

import numpy as np

SHAPES = ("256x256", "128x128", "64x64", "32x128", "256x256 each")
PRODUCTS = ("y", "dx", "dw", "gated", "int8", "int8 gated")   # N, K of linear; gated: I, H

# (product, groups, rows, N, K): shape.  256 x 256 tiles of y and dw by blocks that
# stay: one tile a block, several of one chunk, of two and of many, wide and ragged.
# Those of dx and gated, and of y by a block for each ("each"), have last tiles of
# every height.
SIZES = {
    ("y", 1, 5, 72, 72): "32x128",
    ("y", 7, 900, 1000, 201): "32x128",
    ("y", 3, 65, 1000, 520): "64x64",
    ("y", 300, 12000, 72, 72): "128x128",
    ("y", 5, 3333, 4100, 1100): "128x128",
    ("y", 130, 39000, 136, 72): "256x256",
    ("y", 40, 12000, 520, 520): "256x256",
    ("y", 20, 9000, 1033, 1100): "256x256",
    ("y", 1, 9000, 4100, 1100): "256x256",
    ("y", 40, 5120, 1033, 520): "256x256 each",
    ("dx", 1, 3, 72, 72): "32x128",
    ("dx", 3, 65, 520, 72): "64x64",
    ("dx", 300, 12000, 72, 72): "128x128",
    ("dx", 40, 12000, 520, 520): "256x256",
    ("dx", 21, 9001, 500, 1033): "256x256",
    ("dw", 1, 1, 72, 72): "256x256",
    ("dw", 700, 14000, 264, 300): "256x256",
    ("dw", 40, 9000, 1033, 520): "256x256",
    ("dw", 40, 9000, 1034, 520): "256x256",
    ("dw", 300, 300, 72, 72): "128x128",
    ("dw", 7, 5000, 520, 391): "64x64",
    ("gated", 1, 7, 72, 72): "32x128",
    ("gated", 3, 100, 500, 520): "64x64",
    ("gated", 130, 9100, 72, 72): "128x128",
    ("gated", 40, 5200, 520, 201): "256x256",
    ("gated", 9, 5000, 1033, 523): "256x256",
    ("int8", 1, 9, 72, 72): "32x128",
    ("int8", 40, 5200, 264, 72): "64x64",
    ("int8", 300, 12000, 72, 72): "128x128",
    ("int8", 130, 39000, 136, 200): "256x256",
    ("int8", 20, 9000, 1033, 2100): "256x256",
    ("int8", 40, 5120, 1033, 520): "256x256 each",
    ("int8 gated", 1, 5, 72, 72): "32x128",
    ("int8 gated", 40, 5200, 136, 72): "64x64",
    ("int8 gated", 130, 9100, 72, 72): "128x128",
    ("int8 gated", 40, 5200, 520, 520): "256x256",
    ("int8 gated", 40, 5200, 521, 1100): "256x256",
}


def shape(lib, product, G, R, N, K):
    f = lib.dsmoe_grouped_shape
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    i = f(PRODUCTS.index(product), G, R, N, K)
    return SHAPES[i] if i >= 0 else None


def group_sizes(G, R):
    """G sizes that sum to R: uneven, some 0, some of one row or a whole tile."""
    r = np.random.default_rng(G + R)
    w = r.random(G) ** 2
    if G > 2:
        w[r.integers(0, G, G // 6)] = 0
    s = np.floor(w / w.sum() * R).astype(int)
    for i, n in enumerate((1, 256, 64, 65)):
        if G > 8 * (i + 1):
            s[8 * i + 3] = min(n, R // G * 2)
    while s.sum() > R:
        s[s.argmax()] -= s.sum() - R if s.max() > s.sum() - R else s.max()
    s[s.argmax()] += R - s.sum()
    return s.tolist()
