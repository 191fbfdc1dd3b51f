"""The index arithmetic of csrc/cache_index.h, compiled for the host: tiles,
the cut of the step stream, partial-result slots and joins, page lookups."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "cache_index.h"
using namespace attn25;
extern "C" {
void tiles(int G, int T, int* o) { RowTiles r = row_tiles(G, T); o[0]=r.head_tile; o[1]=r.tok_tile; o[2]=r.rows;
  o[3]=r.head_chunks; o[4]=r.tok_tiles; o[5]=r.tiles; o[6]=tree_groups(r.tiles); }
int steps(int len, int n, int has) { return item_steps(len, n, has != 0); }
long long raw(long long t, int gs, int g) { return raw_cut(t, gs, g); }
long long snap(long long at, long long a, long long b) { return snapped(at, a, b); }
void inner(long long t, int gs, long long a, long long b, int* o) { InnerCuts c = inner_cuts(t, gs, a, b); o[0]=c.first; o[1]=c.count; }
int even(int s, int k, int n) { return even_cut(s, k, n); }
long long muldiv(long long x, int y, long long z) { return mul_div(x, y, z); }
int page(const int* tab, int P, int n, int b, int i) { CacheIndex c{tab, nullptr, 4, 1, P, 16, n, n*16}; return page_at(c, b, i); }
long long entry(int H, int cap, int b, int h, int s) { CacheIndex c{nullptr, nullptr, 1<<16, H, 1, cap, 1, cap}; return slot_entry(c, b, h, s); }
int clamp(int raw, int most, int* bad) { bool x = false; int r = clamp_count(raw, most, x); *bad = x; return r; }
int size_ok(int ps) { return page_size_ok(ps); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("cache_index")
    src = d / "x.cpp"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "tiled_attention_25_b200", "csrc"), str(src), "-o", str(d / "x.so")], check=True)
    lib = ctypes.CDLL(str(d / "x.so"))
    ll, i = ctypes.c_longlong, ctypes.c_int
    for f in (lib.raw, lib.entry, lib.snap, lib.muldiv):
        f.restype = ll
    lib.raw.argtypes, lib.snap.argtypes, lib.muldiv.argtypes = [ll, i, i], [ll, ll, ll], [ll, i, ll]
    lib.inner.argtypes = [ll, i, ll, ll, ctypes.c_void_p]
    return lib


def tiles(lib, G, T):
    o = (ctypes.c_int * 7)()
    lib.tiles(G, T, o)
    return list(o)


def test_tiles_cover_every_row_once(lib):
    for G in (1, 2, 3, 4, 5, 7, 8, 16, 40, 127, 128, 129, 200, 256, 300):
        for T in (1, 2, 3, 8, 33, 100, 128, 129, 1024):
            ht, tt, rows, hc, tts, n, groups = tiles(lib, G, T)
            assert rows == ht * tt <= 128 and n == hc * tts and ht <= 128 and tt <= 128
            seen = set()
            for tile in range(n):
                t0, h0 = tile // hc * tt, tile % hc * ht
                for r in range(rows):
                    tok, head = t0 + r // ht, h0 + r % ht
                    if tok < T and head < G:
                        assert (tok, head) not in seen
                        seen.add((tok, head))
            assert len(seen) == G * T
            assert groups >= 1 and (groups == 1 or groups * n <= 148)


def test_the_cut_covers_the_stream_and_every_cut_item_is_joined(lib):
    rng = np.random.default_rng(0)
    for _ in range(400):
        B, H = int(rng.integers(1, 30)), int(rng.integers(1, 9))
        lens = rng.integers(0, rng.choice([3, 300, 4000, 100000]), size=B)
        cnt = rng.integers(0, 4, size=B)
        has = int(rng.integers(0, 2))
        st = [lib.steps(int(a), int(c), has) for a, c in zip(lens, cnt)]
        items, total = [], 0
        for b in range(B):
            for _ in range(H):
                if st[b]:
                    items.append((total, total + st[b]))
                    total += st[b]
        groups = int(rng.choice([1, 2, 7, 148]))
        if total == 0 or len(items) <= groups:
            continue  # one piece to a group instead
        cuts = [0]
        for g in range(1, groups):
            at = lib.raw(total, groups, g)
            i0, i1 = next(x for x in items if x[0] <= at < x[1])
            cuts.append(lib.snap(at, i0, i1))
        cuts.append(total)
        assert cuts == sorted(cuts)
        slots, counters = [], []
        for i0, i1 in items:
            pieces = []  # (slot, begin, end) as the groups write them
            out = (ctypes.c_int * 2)()
            lib.inner(total, groups, i0, i1, out)
            first, count = out
            for g in range(groups):
                s, e = max(i0, cuts[g]), min(i1, cuts[g + 1])
                if s < e:
                    pieces.append((2 * g if s > i0 else 2 * first - 1, s, e))
            assert sum(e - s for _, s, e in pieces) == i1 - i0
            if len(pieces) == 1:
                continue
            # what a piece's record says of its item: the pieces and their slots, the counter
            assert len(pieces) == count + 1
            assert [x[0] for x in pieces] == [2 * first - 1] + [2 * (first + k) for k in range(count)]
            assert all(e - s >= 4 for _, s, e in pieces)
            slots += [x[0] for x in pieces]
            counters.append(first)
        # a slot is written by one piece at most, and fits the workspace
        assert len(slots) == len(set(slots)) and all(0 <= s < 2 * groups for s in slots)
        assert len(counters) == len(set(counters)) and all(0 <= c < groups for c in counters)


def test_even_pieces_cover_an_item(lib):
    for s in (1, 2, 5, 33, 8200):
        for n in range(1, min(s, 148) + 1):
            cuts = [lib.even(s, k, n) for k in range(n + 1)]
            sizes = [b - a for a, b in zip(cuts, cuts[1:])]
            assert cuts[0] == 0 and cuts[-1] == s and min(sizes) >= 1 and max(sizes) == -(-s // n)


def test_products_in_32_and_64_bits(lib):
    for x in (0, 1, 5, (1 << 24) - 1, 1 << 24, 535000000):
        for y in (1, 7, 148):
            for z in (1, 13, (1 << 24) - 1, 1 << 24, 535000000):
                assert lib.muldiv(x, y, z) == x * y // z


def test_steps(lib):
    assert [lib.steps(*x) for x in ((0, 0, 1), (500, 0, 1), (0, 1, 0), (0, 1, 1), (1, 1, 0), (128, 1, 1), (129, 129, 1))] == \
        [0, 0, 1, 1, 1, 2, 4]


def test_pages_outside_the_pool(lib):
    tab = (ctypes.c_int * 12)(0, 4, 5, -1, 1 << 30, -(1 << 31), 3, 2, 1, 0, 0, 0)
    assert [lib.page(tab, 5, 3, b, i) for b in range(3) for i in range(3)] == [0, 4, -1, -1, -1, -1, 3, 2, 1]
    assert [lib.page(None, 5, 3, b, i) for b in range(2) for i in range(3)] == [0, 1, 2, 3, 4, -1]


def test_entries_and_counts(lib):
    assert lib.entry(8, 1 << 20, 65535, 7, 5) == (65535 * 8 + 7) * (1 << 20) + 5  # beyond 32 bits
    bad = ctypes.c_int()
    got = []
    for raw in (-5, 0, 3, 7, 8, 1 << 30):
        got.append((lib.clamp(raw, 7, ctypes.byref(bad)), bad.value))
    assert got == [(0, 1), (0, 0), (3, 0), (7, 0), (7, 1), (7, 1)]
    assert [ps for ps in range(1, 600) if lib.size_ok(ps)] == [16, 32, 64, 128, 256, 384, 512]
