"""The checks of the lists that the chunk attention keeps in its workspace (csrc/chunk_list.h), built for
the host: what they let through stays inside the call's sizes, whatever the workspace holds, and
every list that a plan writes is let through."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_long_kap_b200", "csrc")

SOURCE = r"""
#include "chunk_list.h"
using namespace cosa;
extern "C" {
int plan(const ChunkBounds* n, int tiles, long long units) { return plan_fits(*n, tiles, units); }
int tile(const ChunkBounds* n, const ChunkTile* t, long long at, int hk) { return tile_fits(*n, *t, at, hk); }
int join(const ChunkBounds* n, int ntok, int tok0, int hk, int first, int last) {
  return join_fits(*n, ntok, tok0, hk, first, last);
}
// Walks a share; the lengths change from nb0 to nb1 before step `when`.  Returns the segments taken
// (-1: outside what the lengths at that moment allow), *blocks their sum, *lost whether it broke off.
int walk(int batch, int heads, const int* nb0, const int* nb1, int when, int b0, int off, int hk, long long left,
         long long* blocks, int* lost) {
  DecodeWalk w;
  w.left = left, w.hk = hk, w.b = b0, w.off = off, w.lost = false, w.have = true;
  int step = 0;
  auto tile_of = [&](int b) {
    ChunkTile t = {};
    t.b = b, t.jb = 5, t.nb = (step < when ? nb0 : nb1)[b];
    return t;
  };
  w.tile = tile_of(b0);
  *blocks = 0;
  for (; w.next(batch, heads, tile_of); w.advance(batch), ++step) {
    if (w.b < 0 || w.b >= batch || w.hk >= heads || w.nb < 1 || w.jb < 5 || w.jb + w.nb > 5 + w.tile.nb) return -1;
    *blocks += w.nb;
  }
  *lost = w.lost;
  return step;
}
}
"""

INTS = (-2**31, -1000, -1, 0, 1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 127, 128, 129, 1000, 2**30, 2**31 - 1)


class Bounds(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "total_q", "max_kv", "num_kv_heads", "span", "max_tiles", "ctas")]


class Tile(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tok0", "ntok", "pos0", "b", "jb", "nb", "kv", "prefix")]


@pytest.fixture(scope="module")
def lists(tmp_path_factory):
    d = tmp_path_factory.mktemp("lists")
    (d / "lists.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-shared", "-fPIC",
                    "-I", CSRC, "-o", str(d / "lists.so"), str(d / "lists.cpp")], check=True)
    L = ctypes.CDLL(str(d / "lists.so"))
    L.plan.argtypes = [ctypes.POINTER(Bounds), ctypes.c_int, ctypes.c_longlong]
    L.tile.argtypes = [ctypes.POINTER(Bounds), ctypes.POINTER(Tile), ctypes.c_longlong, ctypes.c_int]
    L.join.argtypes = [ctypes.POINTER(Bounds)] + [ctypes.c_int] * 5
    return L


N = Bounds(batch=3, total_q=33, max_kv=1000, num_kv_heads=2, span=16, max_tiles=5, ctas=148)


def test_what_passes_stays_inside(lists):
    rng = random.Random(1)
    passed = 0
    for _ in range(200000):
        v = [rng.randrange(0, 34), rng.randrange(1, 17), 0, rng.randrange(3), rng.randrange(8), rng.randrange(1, 5),
             rng.randrange(1, 1001), 0, rng.randrange(6), rng.randrange(2)]
        for i in range(10):
            if rng.random() < 0.1:
                v[i] = rng.choice(INTS)
        t, at, hk = Tile(*v[:8]), v[8] << rng.choice((0, 0, 0, 32)), v[9]
        if lists.tile(N, t, at, hk):
            passed += 1
            assert 0 <= t.tok0 and 1 <= t.ntok <= 16 and t.tok0 + t.ntok <= 33
            assert 0 <= t.b < 3 and 0 <= hk < 2 and 1 <= t.kv <= 1000
            assert 0 <= t.jb and 1 <= t.nb and (t.jb + t.nb - 1) * 128 < t.kv
            assert 0 <= at < t.nb + 2
    assert passed > 1000
    for _ in range(200000):
        ntok, tok0, hk, last = (rng.choice(INTS) for _ in range(4))
        first = rng.randrange(148)
        if lists.join(N, ntok, tok0, hk, first, last):
            assert 1 <= ntok <= 16 and 0 <= tok0 <= 33 - ntok and 0 <= hk < 2 and first < last < 148
    for tiles in INTS:
        for units in INTS + (2**62, -2**62):
            if lists.plan(N, tiles, units):
                assert 0 <= tiles <= 5 and 0 <= units <= tiles * (8 + 2)


def test_what_a_plan_writes_passes(lists):
    assert lists.plan(N, 0, 0) and lists.plan(N, 5, 50) and lists.plan(N, 1, 3)
    for kv in (1, 127, 128, 129, 1000):
        blocks = -(-kv // 128)
        for jb in range(blocks):
            for nb in range(1, blocks - jb + 1):
                for at in range(nb + 2):
                    for tok0, ntok in ((0, 1), (0, 16), (17, 16), (32, 1)):
                        assert lists.tile(N, Tile(tok0, ntok, 0, 2, jb, nb, kv, 0), at, 1)
    for last in (1, 147):
        assert lists.join(N, 16, 17, 1, 0, last)
    assert lists.join(N, 1, 32, 0, 146, 147)
    wide = Bounds(4096, 1 << 30, 1 << 30, 65535, 256, 1 << 30, 148)
    assert lists.tile(wide, Tile((1 << 30) - 256, 256, 0, 4095, 0, 1 << 23, 1 << 30, 0), (1 << 23) + 1, 65534)
    assert lists.plan(wide, 1 << 30, (1 << 30) * ((1 << 23) + 2))


def _walk(L, nb0, nb1, when, b0, off, hk, left, heads=2):
    n = len(nb0)
    arr = ctypes.c_int * n
    blocks, lost = ctypes.c_longlong(0), ctypes.c_int(0)
    steps = L.walk(n, heads, arr(*nb0), arr(*nb1), when, b0, off, hk, ctypes.c_longlong(left), ctypes.byref(blocks),
                   ctypes.byref(lost))
    return steps, blocks.value, bool(lost.value)


def test_a_share_is_walked_to_its_end(lists):
    nb = [3, 0, 1, 7, 0]
    order = [(h, b, j) for h in range(2) for b in range(5) for j in range(nb[b])]
    for i, (h, b, j) in enumerate(order):
        for left in range(1, len(order) - i + 1):
            steps, blocks, lost = _walk(lists, nb, nb, 99, b, j, h, left)
            assert blocks == left and not lost and steps == len({x[:2] for x in order[i:i + left]})


@pytest.mark.parametrize("after", [[0, 0, 0, 0, 0], [1, 0, 0, 0, 0], [3, 0, 1, 2, 0], [9, 9, 9, 9, 9]])
def test_a_share_ends_though_its_lengths_change_under_it(lists, after):
    """Lengths gone to nothing kept the walk from ever ending."""
    nb = [3, 0, 1, 7, 0]
    order = [(h, b, j) for h in range(2) for b in range(5) for j in range(nb[b])]
    for i, (h, b, j) in enumerate(order):
        for when in range(3):
            steps, blocks, lost = _walk(lists, nb, after, when, b, j, h, len(order) - i)
            assert steps >= 0 and blocks <= len(order) - i and (lost or blocks == len(order) - i)
