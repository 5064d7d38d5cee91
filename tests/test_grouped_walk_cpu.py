"""The blocks that stay (csrc/grouped_stream.h) on the CPU: which tiles each takes, by the code that the kernel runs
(dsmoe_grouped_walk, not part of the interface), and how far its copies may be ahead of its products."""

import ctypes

import numpy as np
import pytest

ROWS = COLS = 256
CHUNK = 64


@pytest.fixture(scope="module")
def lib():
    import fp8_block_scaled_dsmoe_amd as d
    f = d.lib.dsmoe_grouped_walk
    f.restype = ctypes.c_int64
    f.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                  ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int64]
    return d.lib


def _walk(lib, dw, offsets, R, N, K, blocks, most=4096):
    """Tiles [n][7] of each block."""
    off = None if offsets is None else np.asarray(offsets, np.int32)
    got = []
    for b in range(blocks):
        out = np.zeros((most, 7), np.int32)
        n = lib.dsmoe_grouped_walk(dw, None if off is None else off.ctypes.data, 1 if off is None else off.size - 1, R, N, K, b,
                                   blocks, out.ctypes.data, most)
        assert 0 <= n <= most
        got.append(out[:n])
    return got


def _sizes(r, G):
    s = r.integers(0, 700, G)
    s[r.random(G) < 0.3] = 0
    s[r.integers(0, G)] = r.choice([1, 255, 256, 257, 5000])
    return s


CASES = [(0, 1, 8), (1, 1, 8), (2, 3, 64), (3, 40, 256), (4, 300, 256), (5, 1024, 256), (6, 70, 16)]


@pytest.mark.parametrize("seed,G,blocks", CASES)
@pytest.mark.parametrize("N,K", [(1, 1), (256, 64), (257, 65), (1033, 520), (520, 4000)])
def test_every_tile_once(lib, seed, G, blocks, N, K):
    sizes = _sizes(np.random.default_rng(seed), G)
    off = np.concatenate([[0], np.cumsum(sizes)])
    R = int(off[-1]) + seed % 3      # rows behind the last group too
    y = np.concatenate(_walk(lib, 0, off, R, N, K, blocks))
    want = [(g, off[g] + m, off[g + 1], n, 0, 0, -(-K // CHUNK)) for g in range(G) for m in range(0, sizes[g], ROWS)
            for n in range(0, N, COLS)]
    assert sorted(map(tuple, y.tolist())) == sorted(want)
    dw = np.concatenate(_walk(lib, 1, off, R, N, K, blocks, most=8192))
    want = [(g, m, N, n, off[g], off[g + 1], max(1, -(-sizes[g] // CHUNK))) for g in range(G) for m in range(0, N, ROWS)
            for n in range(0, K, COLS)]
    assert sorted(map(tuple, dw.tolist())) == sorted(want)


def test_one_group_without_offsets(lib):
    y = np.concatenate(_walk(lib, 0, None, 1000, 300, 70, 64))
    assert sorted(map(tuple, y.tolist())) == sorted((0, m, 1000, n, 0, 0, 2) for m in (0, 256, 512, 768) for n in (0, 256))


@pytest.mark.parametrize("seed", range(8))
def test_offsets_that_break_the_rule(lib, seed):
    """Every tile stays within the operands, and the walk ends."""
    r = np.random.default_rng(seed)
    G, R, N, K = 24, 3000, 520, 300
    bad = r.integers(-R, 2 * R, G + 1)
    if seed % 2:
        bad[r.integers(0, G + 1, 9)] = r.choice([-2 ** 31, 2 ** 31 - 1, R, 0], 9)
    y = np.concatenate(_walk(lib, 0, bad, R, N, K, 64))
    assert ((0 <= y[:, 1]) & (y[:, 1] < y[:, 2]) & (y[:, 2] <= R) & (0 <= y[:, 3]) & (y[:, 3] < N)).all()
    dw = np.concatenate(_walk(lib, 1, bad, R, N, K, 64))
    assert ((0 <= dw[:, 1]) & (dw[:, 1] < N) & (0 <= dw[:, 3]) & (dw[:, 3] < K)).all()
    assert ((0 <= dw[:, 4]) & (dw[:, 4] <= dw[:, 5]) & (dw[:, 5] <= R)).all()
    assert (dw[:, 6] == np.maximum(1, -(-(dw[:, 5] - dw[:, 4]) // CHUNK))).all()


def _schedule(chunks):
    """A block's loop over tiles of these chunks, as grouped_stream_kernel has it: (the most tiles entered past the
    products', the (tile, chunk) of every product's four halves)."""
    state = {"entered": 0, "left": 0, "ahead": 0}
    source, stage, done = dict.fromkeys(("a0", "a1", "b0", "b1")), ({}, {}), 0

    def enter():
        some = state["entered"] < len(chunks)
        tile = state["entered"] if some else None       # past the last: zeros
        state["left"] = chunks[tile] if some else 1 << 30
        state["entered"] += some
        state["ahead"] = max(state["ahead"], state["entered"] - done - 1)
        for k in source:
            source[k] = [tile, 0]

    def copy(s, *halves):
        for k in halves:
            stage[s][k] = tuple(source[k])
            source[k][1] += 1

    enter()
    copy(0, "b0", "a0", "b1", "a1")
    state["left"] -= 1
    if state["left"] == 0:
        enter()
    copy(1, "b0", "a0", "b1")
    state["left"] -= 1
    seen, st, products = [], 0, chunks[0]
    b0 = stage[0]["b0"]
    while True:
        nx = 1 - st
        halves = [b0, stage[st]["a0"], stage[st]["b1"]]
        copy(nx, "a1")
        if state["left"] == 0:
            enter()
        copy(st, "b0")
        halves.append(stage[st]["a1"])
        b0 = stage[nx]["b0"]
        copy(st, "a0", "b1")
        state["left"] -= 1
        seen.append(halves)
        st = nx
        products -= 1
        if products == 0:
            done += 1
            if done >= state["entered"]:
                return state["ahead"], seen
            products = chunks[done]


def test_copies_ahead_of_the_products(lib):
    """Whatever the tiles' chunks, the products find the halves of their chunk, and no more tiles are entered ahead of them
    than the kernel's queue is sized by (which tiles of one chunk need)."""
    r = np.random.default_rng(0)
    worst = 0
    for _ in range(2000):
        chunks = r.choice([1, 1, 1, 2, 3, 5, 9], r.integers(1, 13)).tolist()
        ahead, seen = _schedule(chunks)
        assert seen == [[(i, c)] * 4 for i, n in enumerate(chunks) for c in range(n)]
        worst = max(worst, ahead)
    assert worst == lib.dsmoe_grouped_walk_ahead()


def test_when_blocks_stay(lib):
    """y in 256 x 256 tiles: a block for each tile up to 192 rows per group, and up to 224 where there are at most four
    tiles a CU, as measured; blocks that stay past that."""
    import grouped_kernels as gk
    for product in ("y", "int8"):
        for G, N, K, rows in ((256, 7168, 2048, 192), (64, 7168, 2048, 160), (64, 1024, 512, 208), (32, 2048, 7168, 224)):
            assert gk.shape(lib, product, G, G * rows, N, K) == "256x256 each", (G, N, K, rows)
        for G, N, K, rows in ((256, 7168, 2048, 208), (256, 7168, 2048, 224), (64, 7168, 2048, 208), (256, 2048, 512, 224),
                              (32, 4096, 4096, 320)):
            assert gk.shape(lib, product, G, G * rows, N, K) == "256x256", (G, N, K, rows)
