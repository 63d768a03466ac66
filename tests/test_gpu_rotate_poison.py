"""Cached 8-bit keys that hold infinities, NaNs or nothing, turned on the GPU."""
import math

import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from tests import rotate_ref as R
from tests.test_gpu_rotate import (BLOCK, DIM, KIND, _errors, _lib, check_moved,  # noqa: F401
                                   filled_pool, ok, tables_of)

pytestmark = pytest.mark.gpu


def set_scale(pool, block, h, row, value):
    at = BLOCK * DIM + 4 * row
    pool[block, h, at:at + 4] = torch.tensor([value]).view(torch.uint8).cuda()


@pytest.mark.parametrize("r,side", [(128, False), (128, True), (64, False), (30, False)])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_an_overflowed_key_stays_one(fmt, r, side):
    # a row whose scale is infinite or NaN gives NaN scores before the turn and after it
    g = torch.Generator().manual_seed(17)
    lens = [40]
    tables, blocks = tables_of(g, lens)
    pool = filled_pool(g, blocks, 2, fmt)
    bad = {3: math.inf, 17: math.nan, 38: -math.inf}
    for i, value in bad.items():
        set_scale(pool, int(tables[0, i // BLOCK]), 1, i % BLOCK, value)
    # and one that an infinity in a row left: scale infinite, codes 0 beside it
    at = int(tables[0, 1]), 1, 5
    pool[at[0], at[1], at[2] * DIM:(at[2] + 1) * DIM] = 0
    set_scale(pool, *at, math.inf)
    bad[21] = math.inf
    before = pool.clone()
    shifts = torch.tensor([-9], dtype=torch.int32).cuda()
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                       B.make_rotation(r, interleaved=side), shifts=shifts, kv_format=KIND[fmt])
    ok()
    new = R.tiles_values(pool.cpu(), fmt)
    for i in bad:
        row = new[int(tables[0, i // BLOCK]), 1, i % BLOCK]
        assert (~torch.isfinite(row)).any()
        assert not math.isfinite(float(row @ torch.ones(DIM, dtype=torch.float64)))
        # (a healthy stand-in, so that the rest can be compared)
        for p in (before, pool):
            b, h, o = int(tables[0, i // BLOCK]), 1, i % BLOCK
            p[b, h, o * DIM:(o + 1) * DIM] = 0
            set_scale(p, b, h, o, 0.0)
    by = [[torch.full((40,), -9)] * 2]
    check_moved(before, pool, tables, lens, by, R.theta(r)[0], side, fmt)


@pytest.mark.parametrize("whole", [False, True])
def test_fp8_codes_that_are_nans_stay_nans(whole):
    g = torch.Generator().manual_seed(18)
    tables, blocks = tables_of(g, [16])
    pool = filled_pool(g, blocks, 1, "fp8")
    b = int(tables[0, 0])
    if whole:
        pool[b, 0, 2 * DIM:3 * DIM] = 0x7F
    else:
        pool[b, 0, 2 * DIM + 9] = 0xFF
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor([16], dtype=torch.int32).cuda(),
                       B.make_rotation(128), shifts=torch.tensor([5], dtype=torch.int32).cuda(),
                       kv_format=B.PA_KV_FP8)
    ok()
    got = R.tiles_values(pool.cpu(), "fp8")[b, 0]
    want = torch.zeros(16, DIM, dtype=torch.bool)
    want[2] = True
    if not whole:
        want[2] = False
        want[2, 9] = want[2, 9 + 64] = True
    assert torch.equal(torch.isnan(got), want)
    assert torch.isfinite(got[~want]).all()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_keys_of_zeros_and_of_extreme_scales(fmt):
    # the largest and smallest scales: codes are turned by themselves, so that neither
    # overflows or vanishes on the way
    g = torch.Generator().manual_seed(19)
    tables, blocks = tables_of(g, [16])
    pool = filled_pool(g, blocks, 1, fmt)
    b = int(tables[0, 0])
    scales = [2.0 ** k for k in (-120, -100, -60, -20, 0, 20, 60, 100, 110, 116)]
    for row, s in enumerate(scales):
        set_scale(pool, b, 0, row, s)
    pool[b, 0, 12 * DIM:13 * DIM] = 0                     # a key of zeros
    before = pool.clone()
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor([16], dtype=torch.int32).cuda(),
                       B.make_rotation(128), shifts=torch.tensor([77], dtype=torch.int32).cuda(),
                       kv_format=KIND[fmt])
    ok()
    check_moved(before, pool, tables, [16], [[torch.full((16,), 77)]], R.theta(128)[0], False, fmt)
    row = R.tiles_values(pool.cpu(), fmt)[b, 0, 12]
    assert (row == 0).all()
