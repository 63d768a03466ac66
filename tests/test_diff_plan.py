"""Sizes of differential attention's launches, compiled for the host."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_decode_18_gb300", "csrc")
HOST = r"""
#include "pa_diff_plan.h"
extern "C" void merge(int by_row, long long longest, int qt, int g, int* out) {
  const pa::DiffMerge m = pa::diff_merge(by_row != 0, longest, qt, g);
  out[0] = m.warps, out[1] = m.chunk, out[2] = m.chunks;
}
extern "C" long long pairs(long long s, long long t, long long longest, int unit) {
  return pa::diff_pairs(s, t, longest, unit);
}
extern "C" long long warp_longest(long long max_q_len, int min_lq) {
  return pa::diff_warp_longest(max_q_len, min_lq);
}
extern "C" int fit(long long pairs, long long heads, long long tiles, int start_cost4) {
  return pa::diff_tiles_fit(pairs, heads, tiles, start_cost4);
}
extern "C" void deal(int warps, int nrows, int warp, int* out) {
  const pa::DiffDeal d = pa::diff_deal(warps, nrows, warp);
  out[0] = d.row, out[1] = d.group, out[2] = d.per_row;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("diff_plan")
    src, lib = d / "plan.cc", d / "plan.so"
    src.write_text(HOST)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-ftrapv", "-I", CSRC,
                    "-o", str(lib), str(src)], check=True)
    lib = ctypes.CDLL(str(lib))
    i64 = ctypes.c_longlong
    lib.pairs.restype = lib.warp_longest.restype = i64
    lib.fit.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.pairs.argtypes, lib.warp_longest.argtypes = [i64, i64, i64, ctypes.c_int], [i64, ctypes.c_int]
    return lib


def three(fn, *args):
    out = (ctypes.c_int * 3)()
    fn(*args, out)
    return tuple(out)


@pytest.mark.parametrize("by_row", [0, 1])
@pytest.mark.parametrize("G", range(1, 9))
def test_a_merge_has_a_warp_for_every_row(plan, by_row, G):
    # The bound of the windows sizes the launch, the device's windows say how many rows
    # there are: whatever they say, no row of a CTA is without a warp, since a row's
    # warps are what its loop over the pieces steps by.
    QT = 8 // G
    for longest in (1, 2, 3, 4, 7, 8, 9, 40, 1 << 40):
        warps, chunk, chunks = three(plan.merge, by_row, ctypes.c_longlong(longest), QT, G)
        assert warps in (4, 8) and 1 <= chunk <= warps
        assert chunk * chunks >= min(longest, QT) * G    # rows that the call announces
        for found in range(1, QT + 1):                   # tokens that the device finds in a tile
            nrows = min(chunk, found * G)
            got = [three(plan.deal, warps, nrows, w) for w in range(warps)]
            for row, group, per_row in got:
                assert per_row >= 1 and 0 <= group < per_row
            for row in range(nrows):
                assert sorted(g for r, g, _ in got if r == row) == list(range(got[0][2]))


def test_a_plan_holds_the_windows_that_come_to_it(plan):
    # the warp tiles' plan: of a batch with longer windows, which the tcgen05 tiles take, the
    # short ones alone
    rng = random.Random(3)
    for _ in range(300):
        G = rng.randint(1, 8)
        QT, min_lq = 8 // G, -(-32 // G)
        qs = [rng.randint(0, rng.choice([3, 40, 400])) for _ in range(rng.randint(1, 60))]
        longest, T = max(qs), sum(qs) + rng.choice([0, 0, 50])
        cap = plan.pairs(len(qs), T, plan.warp_longest(longest, min_lq), QT)
        assert sum(-(-n // QT) for n in qs if n < min_lq) <= cap <= len(qs) * -(-(min_lq - 1) // QT)
        unit = 2 * (128 // G)
        assert sum(-(-n // unit) for n in qs) <= plan.pairs(len(qs), T, longest, unit)


@pytest.mark.parametrize("G,seqs,total,longest", [(8, 81, 20250, 330), (8, 8, 16700, 4000),
                                                  (4, 8, 33400, 8000), (2, 8, 66800, 16000),
                                                  (1, 8, 1 << 20, 1 << 18)])
def test_long_windows_take_no_room_in_the_plan_of_short_ones(plan, G, seqs, total, longest):
    # beside the ring of 160 KB a plan has some 16,600 words: a word a pair, three a sequence
    cap = plan.pairs(seqs, total, plan.warp_longest(longest, -(-32 // G)), 8 // G)
    assert cap + 3 * seqs + 3 < 1000


def test_flat_tiles_stay_in_32_bits(plan):
    # (-ftrapv: the check itself must not wrap)
    rng = random.Random(4)
    for _ in range(4000):
        pairs, heads = rng.randint(1, 1 << 22), rng.randint(1, 1 << 24)
        tiles, cost = rng.randint(0, 1 << 26) >> rng.randint(0, 20), rng.choice([6, 20])
        want = pairs * heads * tiles < 1 << 31 and heads * (4 * tiles + cost) < 1 << 31
        assert bool(plan.fit(pairs, heads, tiles, cost)) == (want or tiles == 0)
    # thousands of sequences over one long prefix, many heads; the batches of the tests
    assert not plan.fit(4096, 16, 1 << 16, 6)
    assert not plan.fit(1, 8, 1 << 26, 6)
    assert plan.fit(4096, 4, 1 << 16, 6) and plan.fit(4096, 16, 8192, 6)
    assert plan.fit(1 << 20, 8, 0, 20)
