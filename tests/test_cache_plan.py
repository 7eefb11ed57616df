"""The index arithmetic of the attention over the paged cache
(csrc/cache_plan.h), compiled for the host and compared with brute force."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "cache_plan.h"
using namespace dsvit;
extern "C" {
void blocks(int p0, int p1, int window, int sinks, int shift, int* out) {
  const KeyBlocks b = key_blocks(p0, p1, window, sinks, shift);
  out[0] = b.sink; out[1] = b.first; out[2] = b.count;
}
int block_at(int p0, int p1, int window, int sinks, int shift, int i) {
  return key_blocks(p0, p1, window, sinks, shift).at(i);
}
int64_t begin(int64_t w, int64_t W, int64_t U) { return deal(U, W).begin(w); }
int refused(int row0, int row1, int kv, int rows, int max_rows, int64_t places) {
  return seq_refused(row0, row1, kv, rows, max_rows, places);
}
int there(int page, int64_t n) { return page_there(page, n); }
int divide(int n, int d) { return fast_div(d)(n); }
int64_t snapped(int64_t x, int64_t i0, int64_t i1, int64_t snap, int64_t cost) {
  return snap_border(x, i0, i1, snap, cost);
}
int64_t owner(int64_t x, int64_t W, int64_t U) { return deal(U, W).owner(x); }
int64_t checks_from(unsigned block, int threads, int thread) { return check_first(block, threads, thread); }
int64_t checks_step(unsigned blocks, int threads) { return check_step(blocks, threads); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    src, lib = str(d / "plan.cpp"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-fPIC", "-shared",
                    "-I", os.path.join(ROOT, "vit_vision_encoder_gb300", "csrc"), src, "-o", lib, "-lubsan"],
                   check=True)
    h = C.CDLL(lib)
    for f in (h.begin, h.owner):
        f.restype, f.argtypes = C.c_int64, [C.c_int64] * 3
    h.snapped.restype, h.snapped.argtypes = C.c_int64, [C.c_int64] * 5
    h.checks_from.restype, h.checks_from.argtypes = C.c_int64, [C.c_uint, C.c_int, C.c_int]
    h.checks_step.restype, h.checks_step.argtypes = C.c_int64, [C.c_uint, C.c_int]
    return h


def test_blocks_are_those_that_some_row_sees(plan):
    rng = random.Random(1)
    for _ in range(4000):
        shift = rng.choice([4, 7])
        c = rng.choice([1, 1, 2, 7, 60])
        kv = rng.randrange(0, 700)
        window = rng.choice([0, 1, 2, 16, 17, 100, 128, 300, 10 ** 9, 2 ** 31 - 1])
        sinks = rng.choice([0, 1, 4, 16, 17, 130, 2 ** 31 - 1])
        p0, p1 = kv - c, kv - 1
        out = (C.c_int * 3)()
        plan.blocks(p0, p1, window, sinks, shift, out)
        got = [plan.block_at(p0, p1, window, sinks, shift, i) for i in range(out[2])]
        lo = max(0, p0 - window + 1) if window else 0
        seen = [j for j in range(kv) if j >= lo or j < sinks]
        assert got == sorted({j >> shift for j in seen}), (p0, p1, window, sinks, shift)


def test_blocks_at_the_ends_of_the_range(plan):
    """No 32-bit overflow at the largest positions, windows and paddings."""
    out = (C.c_int * 3)()
    top = 2 ** 31 - 1
    for p0, p1 in ((-2 ** 30, -1), (-2 ** 30, 5), (top - 1, top - 1), (0, top - 1), (-2 ** 30, top - 1)):
        for window in (0, 1, 4096, top):
            for sinks in (0, 5, top):
                for shift in (4, 7):
                    plan.blocks(p0, p1, window, sinks, shift, out)
                    if p1 < 0:
                        assert out[2] == 0
                        continue
                    lo = max(0, p0 - window + 1) if window else 0
                    first = lo >> shift
                    sink = min(-(-min(sinks, lo) // 2 ** shift), first)
                    assert list(out) == [sink, first, sink + (p1 >> shift) - first + 1]


def test_shares(plan):
    """Every unit has one worker, shares differ by one unit at most and none is
    empty; the largest counts do not overflow."""
    rng = random.Random(2)
    for _ in range(300):
        W = rng.randrange(1, 300)
        U = rng.randrange(W, 3000)
        edge = [plan.begin(w, W, U) for w in range(W + 1)]
        assert edge[0] == 0 and edge[-1] == U
        sizes = [b - a for a, b in zip(edge, edge[1:])]
        assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
        for w in range(W):
            for x in (edge[w], edge[w + 1] - 1):
                assert plan.owner(x, W, U) == w
    U, W = 1024 * 128 * 2 ** 27 + 5, 1216
    for w in (0, 1, 700, 1215):
        x = plan.begin(w, W, U)
        assert x == w * (U // W) + min(w, U % W) and plan.owner(x, W, U) == w
    assert plan.begin(0, 0, 0) == 0


def test_division_by_the_group(plan):
    top = 2 ** 31 - 1
    for d in list(range(1, 129)) + [2 ** 30, top]:
        for q in (0, 1, 2, 77, top // d - 1, top // d):
            for n in (q * d - 1, q * d, q * d + 1, q * d + d - 1):
                if 0 <= n <= top:
                    assert plan.divide(n, d) == n // d, (n, d)
    rng = random.Random(3)
    for _ in range(5000):
        n, d = rng.randrange(top + 1), rng.randrange(1, 129)
        assert plan.divide(n, d) == n // d


def test_snapped_borders(plan):
    """Borders keep their order, move at most `snap` units (or out of an item's
    first `cost`) and never leave their item; a worker between two borders inside one
    item keeps at least a unit, and every part of an item has tiles."""
    rng = random.Random(4)
    cost = 4
    for _ in range(600):
        counts = [rng.randrange(1, 40) + cost for _ in range(rng.randrange(1, 30))]
        ends = [0]
        for c in counts:
            ends.append(ends[-1] + c)
        U = ends[-1]
        W = rng.randrange(1, min(U, 60) + 1)
        snap = min(6, 3 * (U // W) // 8)
        borders = []
        for w in range(W + 1):
            x = plan.begin(w, W, U)
            if x < U:
                i = max(j for j in range(len(counts)) if ends[j] <= x)
                y = plan.snapped(x, ends[i], ends[i + 1], snap, cost)
                assert y in (x, ends[i], ends[i + 1]) and abs(y - x) <= max(snap, cost)
                assert y == ends[i] or y - ends[i] > cost
                x = y
            borders.append(x)
        assert borders[0] == 0 and borders[-1] == U and borders == sorted(borders)
        for i in range(len(counts)):
            inside = [b for b in borders if ends[i] < b < ends[i + 1]]
            assert len(inside) == len(set(inside))


def test_sequences_and_pages_refused(plan):
    """The checks that the kernels make of entries on the device."""
    top = 2 ** 31 - 1
    ok = (10, 14, 100, 20, 4, 160)
    assert plan.refused(*ok[:5], C.c_int64(ok[5])) == 0

    def at(code, **kw):
        f = dict(zip(("row0", "row1", "kv", "rows", "max_rows", "places"), ok))
        f.update(kw)
        assert plan.refused(f["row0"], f["row1"], f["kv"], f["rows"], f["max_rows"], C.c_int64(f["places"])) == code, kw

    for kw in (dict(row0=-1), dict(row1=9), dict(row1=21), dict(row1=15), dict(row0=-top - 1), dict(row1=top),
               dict(row0=top, row1=-top - 1), dict(row0=0, row1=5), dict(row0=9), dict(row0=-2, row1=-1)):
        at(1, **kw)
    for kw in (dict(kv=-1), dict(kv=161), dict(kv=top), dict(kv=-top - 1)):
        at(2, **kw)
    for kw in (dict(kv=0), dict(kv=160), dict(row1=10), dict(row0=14), dict(kv=top, places=2 ** 40), dict(row0=0, row1=0)):
        at(0, **kw)
    for page, n, want in ((0, 1, 1), (1, 1, 0), (-1, 5, 0), (4, 5, 1), (5, 5, 0), (top, 2 ** 33, 1), (-top - 1, 2 ** 33, 0)):
        assert plan.there(page, C.c_int64(n)) == want


def test_sequences_checked_by_a_grid(plan):
    """Every sequence is checked by one thread, and the first and the step stay positive
    up to the grid of the most rows that a call admits (four a block)."""
    for n in (1, 2, 127, 128, 129, 1024):
        for blocks in (1, 2, 3, 8, 9, 1000):
            step = plan.checks_step(blocks, 128)
            mine = [s for b in range(blocks) for t in range(128) for s in range(plan.checks_from(b, 128, t), n, step)]
            assert sorted(mine) == list(range(n))
    most = 2 ** 30 - 1
    for rows in (2 ** 26 - 4, 2 ** 26, 2 ** 27, 2 ** 27 + 4, 2 ** 28, 2 ** 29, most):
        blocks = -(-rows // 4)
        assert plan.checks_step(blocks, 128) == 128 * blocks
        for b in (0, 7, 8, 2 ** 24 - 1, 2 ** 24, 2 ** 25, blocks - 1):
            if b < blocks:
                assert plan.checks_from(b, 128, 127) == 128 * b + 127
