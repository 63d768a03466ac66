"""Sizes of differential attention's launches, compiled for the host."""
import ctypes
import os
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
    return ctypes.CDLL(str(lib))


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
