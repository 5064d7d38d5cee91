"""Sizes that together run every kernel of the dense products in every form
(not collected: no test_ prefix).  What a size runs is asked of the library, so
a change of its rule that takes a size elsewhere fails test_dense_abi_cpu.py."""

import ctypes

SHAPES = ("256x256", "256x192", "128x256", "128x128, 4 stages", "128x128, 2 stages", "64x64")
PRODUCTS = ("y", "dx", "dw", "gated")   # y, dx, dw: M, N, K of linear; gated: M, I, H

# (product, M, N, K): (shape, several splits of K, shape of the second launch)
SIZES = {
    ("y", 1052, 9813, 201): ("256x256", False, None),
    ("y", 2320, 3338, 200): ("256x192", False, None),
    ("y", 1025, 3601, 272): ("128x256", False, None),
    ("y", 1160, 1665, 222): ("128x128, 4 stages", False, None),
    ("y", 1545, 2436, 223): ("128x128, 2 stages", False, None),
    ("y", 72, 72, 200): ("64x64", False, None),
    ("y", 1232, 1608, 6360): ("256x192", True, None),
    ("y", 1224, 800, 6120): ("128x256", True, None),
    ("y", 769, 260, 3859): ("128x128, 4 stages", True, None),
    ("y", 72, 72, 968): ("64x64", True, None),
    ("y", 7187, 3337, 523): ("256x256", False, "256x192"),
    ("y", 2073, 10865, 257): ("256x256", False, "128x256"),
    ("y", 4877, 3493, 397): ("256x256", False, "128x128, 4 stages"),
    ("y", 4624, 7696, 200): ("256x256", False, "128x128, 2 stages"),
    ("y", 2056, 7696, 200): ("256x256", False, "64x64"),
    ("dx", 2322, 200, 4840): ("256x256", False, None),
    ("dx", 1296, 200, 5944): ("256x192", False, None),
    ("dx", 1174, 262, 3216): ("128x256", False, None),
    ("dx", 1284, 202, 1546): ("128x128, 4 stages", False, None),
    ("dx", 3224, 200, 1166): ("128x128, 2 stages", False, None),
    ("dx", 72, 200, 72): ("64x64", False, None),
    ("dx", 1368, 6368, 1504): ("256x192", True, None),
    ("dx", 1101, 6022, 904): ("128x256", True, None),
    ("dx", 261, 3876, 785): ("128x128, 4 stages", True, None),
    ("dx", 72, 968, 72): ("64x64", True, None),
    ("dx", 4626, 516, 5263): ("256x256", False, "256x192"),
    ("dx", 2840, 264, 8176): ("256x256", False, "128x256"),
    ("dx", 10891, 385, 1465): ("256x256", False, "128x128, 4 stages"),
    ("dx", 6216, 200, 5774): ("256x256", False, "128x128, 2 stages"),
    ("dx", 3076, 213, 5129): ("256x256", False, "64x64"),
    ("dw", 203, 1031, 9827): ("256x256", False, None),
    ("dw", 211, 4624, 1682): ("256x192", False, None),
    ("dw", 272, 1568, 2456): ("128x256", False, None),
    ("dw", 200, 1616, 1224): ("128x128, 4 stages", False, None),
    ("dw", 201, 5406, 642): ("128x128, 2 stages", False, None),
    ("dw", 200, 72, 72): ("64x64", False, None),
    ("dw", 17801, 2600, 976): ("256x256", True, None),
    ("dw", 9048, 776, 1224): ("256x192", True, None),
    ("dw", 6097, 1244, 779): ("128x256", True, None),
    ("dw", 3885, 267, 775): ("128x128, 4 stages", True, None),
    ("dw", 13296, 8280, 72): ("128x128, 2 stages", True, None),
    ("dw", 968, 72, 72): ("64x64", True, None),
    ("dw", 538, 4632, 5156): ("256x256", False, "256x192"),
    ("dw", 264, 2608, 8960): ("256x256", False, "128x256"),
    ("dw", 398, 4872, 3526): ("256x256", False, "128x128, 4 stages"),
    ("dw", 200, 2840, 8104): ("256x256", False, "128x128, 2 stages"),
    ("dw", 211, 6805, 2312): ("256x256", False, "64x64"),
    ("gated", 519, 8201, 200): ("256x256", False, None),
    ("gated", 1543, 2504, 200): ("256x192", False, None),
    ("gated", 528, 3280, 264): ("128x256", False, None),
    ("gated", 1104, 904, 200): ("128x128, 4 stages", False, None),
    ("gated", 1288, 1490, 202): ("128x128, 2 stages", False, None),
    ("gated", 72, 72, 200): ("64x64", False, None),
    ("gated", 1157, 833, 6214): ("256x192", True, None),
    ("gated", 769, 613, 5771): ("128x256", True, None),
    ("gated", 324, 323, 3882): ("128x128, 4 stages", True, None),
    ("gated", 72, 72, 968): ("64x64", True, None),
    ("gated", 2720, 4432, 519): ("256x256", False, "256x192"),
    ("gated", 2093, 5424, 260): ("256x256", False, "128x256"),
    ("gated", 4884, 1732, 400): ("256x256", False, "128x128, 4 stages"),
    ("gated", 1550, 7035, 213): ("256x256", False, "128x128, 2 stages"),
    ("gated", 1540, 5016, 212): ("256x256", False, "64x64"),
}


def kernels(lib, product, M, N, K):
    """(shape, several splits of K, shape of the second launch) of a size; "few
    tokens" as the shape for the few-token kernel."""
    f = lib.dsmoe_dense_kernels
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.POINTER(ctypes.c_int64 * 6)]
    out = (ctypes.c_int64 * 6)()
    assert f(PRODUCTS.index(product), M, N, K, ctypes.byref(out)) == 0
    few, shape, splits, cut, rest, _ = out
    return "few tokens" if few else SHAPES[shape], splits > 1, SHAPES[rest] if cut else None
