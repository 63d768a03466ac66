"""Rotary positions on the GPU: of rows, of a step's rows on their way into the
cache, and of keys that the cache holds, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from tests import rotate_ref as R

pytestmark = pytest.mark.gpu

DIM, BLOCK, TILE = 128, 16, 2112
KIND = {"bf16": 0, "int8": 1, "fp8": 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    B.load()


@pytest.fixture(autouse=True)
def _errors():
    B.pa_debug_read_error()
    yield


def ok():
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == 0


def randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def bits(x):
    return x.contiguous().view(torch.int16)


def positions_of(g, T, far=1 << 20):
    p = (torch.rand((T,), generator=g, dtype=torch.float64) * math.log(far)).exp().to(torch.int32)
    if T > 3:
        p[:4] = torch.tensor([0, 1, far, -3])
    return p


# ---------------------------------------------------------------------------
# pa_rotate
# ---------------------------------------------------------------------------

ROWS = [
    # tokens, heads, rotated dimensions, interleaved, map
    (1, 1, 128, False, {}),
    (5, 3, 128, False, {}),
    (37, 16, 128, True, {}),
    (9, 8, 64, False, dict(scaling="linear", factor=4.0)),
    (9, 24, 64, True, dict(base=5e5, scaling="bands", factor=8.0, original_len=8192)),
    (300, 5, 16, False, dict(scaling="base", factor=2.0)),
    (7, 4, 2, False, {}),
    (7, 4, 2, True, {}),
    (7, 9, 30, False, {}),
    (33, 2, 126, False, dict(base=1e6, scaling="ramp", factor=4.0, original_len=32768, high=32.0)),
    (33, 2, 126, True, dict(base=1e6, scaling="ramp", factor=4.0, original_len=32768, high=32.0)),
    (6, 7, 112, False, {}),
    (6, 7, 20, True, {}),
]


@pytest.mark.parametrize("T,H,r,side,kw", ROWS)
@pytest.mark.parametrize("transpose", [False, True])
def test_rows(T, H, r, side, kw, transpose):
    g = torch.Generator().manual_seed(T * 1000 + H * 10 + r)
    x, pos = randn(g, T, H, DIM), positions_of(g, T)
    rot = B.make_rotation(r, interleaved=side, **kw)
    th, m = R.theta(r, **kw)
    ref, err = R.rotate(x, pos[:, None], th, side, m, transpose)
    xd = x.cuda()
    y = torch.full_like(xd, 9.0)
    B.pa_rotate(xd, pos.cuda(), rot, y, transpose=transpose)
    ok()
    got = y.cpu()
    assert ((got.double() - ref).abs() <= R.held_bf16(ref, err)).all()
    assert torch.equal(bits(got[..., r:]), bits(x[..., r:]))      # not rotated: as it was
    assert torch.equal(bits(xd.cpu()), bits(x))
    # in place, and through strided views: the same bits
    B.pa_rotate(xd, pos.cuda(), rot, xd, transpose=transpose)
    ok()
    assert torch.equal(bits(xd.cpu()), bits(got))
    wide = torch.full((T, H + 3, DIM), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:H + 1] = x.cuda()
    turned = torch.full((H, T, DIM), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    B.pa_rotate(wide[:, 1:H + 1], pos.cuda(), rot, turned, transpose=transpose)
    ok()
    assert torch.equal(bits(turned.cpu()), bits(got))
    assert (wide[:, 0] == 5).all() and (wide[:, H + 1:] == 5).all()


def test_rows_between_them_keep_what_they_hold():
    g = torch.Generator().manual_seed(8)
    x, pos = randn(g, 6, 4, DIM).cuda(), positions_of(g, 6).cuda()
    rot = B.make_rotation(128)
    room = torch.full((8, 6, 144), 3.0, dtype=torch.bfloat16, device="cuda")
    y = room[1:7, 1:5, 8:136]
    B.pa_rotate(x, pos, rot, y)
    ok()
    want = torch.empty_like(x)
    B.pa_rotate(x, pos, rot, want)
    ok()
    assert torch.equal(bits(y), bits(want))
    y.fill_(3.0)
    assert (room == 3).all()


@pytest.mark.parametrize("side", [False, True])
def test_a_broadcast_input_and_given_angles(side):
    # one row for all heads (stride 0), angles from the caller, a magnitude
    g = torch.Generator().manual_seed(2)
    x, pos = randn(g, 5, 1, DIM), positions_of(g, 5, 1000)
    th = torch.linspace(-2.0, 9.0, 24, dtype=torch.float64)
    rot = B.make_rotation_from(th, interleaved=side, magnitude=0.75)
    y = torch.empty((5, 6, DIM), dtype=torch.bfloat16, device="cuda")
    B.pa_rotate(x.cuda().expand(5, 6, DIM), pos.cuda(), rot, y)
    ok()
    ref, err = R.rotate(x.expand(5, 6, DIM), pos[:, None], th, side, 0.75)
    assert ((y.cpu().double() - ref).abs() <= R.held_bf16(ref, err)).all()


@pytest.mark.parametrize("side,r", [(False, 128), (True, 128), (False, 90)])
def test_the_transposed_map_is_the_gradient(side, r):
    # against differences of the plain form: f(x) = sum w . rotate(x) is linear
    # in x, so a difference over any step is its slope; and back again where
    # the magnitude is 1
    g = torch.Generator().manual_seed(4)
    x, w, pos = randn(g, 3, 2, DIM), randn(g, 3, 2, DIM), positions_of(g, 3, 5000)
    rot, (th, m) = B.make_rotation(r, interleaved=side), R.theta(r)
    dx = torch.empty((3, 2, DIM), dtype=torch.bfloat16, device="cuda")
    B.pa_rotate(w.cuda(), pos.cuda(), rot, dx, transpose=True)
    ok()
    _, err = R.rotate(w, pos[:, None], th, side, m, True)
    for d in range(DIM):
        step = torch.zeros_like(x).double()
        step[..., d] = 1.0
        up = (R.rotate(x.double() + step, pos[:, None], th, side)[0] * w.double()).sum(-1)
        down = (R.rotate(x.double() - step, pos[:, None], th, side)[0] * w.double()).sum(-1)
        slope = (up - down) / 2
        assert ((dx[..., d].cpu().double() - slope).abs() <=
                R.held_bf16(slope, err[..., d]) + 1e-9).all()
    y = torch.empty_like(dx)
    B.pa_rotate(x.cuda(), pos.cuda(), rot, y)
    B.pa_rotate(y, pos.cuda(), rot, y, transpose=True)
    ok()
    a, b = R.pairs(r, side)
    # two roundings to bf16 of numbers no longer than the pair, and two turns' errors
    off = torch.zeros(3, 2, DIM, dtype=torch.float64)
    size = x[..., a].double().abs() + x[..., b].double().abs()
    off[..., a] = off[..., b] = size * (3 * R.UBF + 4 * R.UCS)
    assert ((y.cpu().double() - x.double()).abs() <= off).all()


def test_infinities_and_nans_stay_in_their_pair():
    g = torch.Generator().manual_seed(5)
    x, pos = randn(g, 4, 2, DIM), torch.tensor([3, 50, 7, 1], dtype=torch.int32)
    x[1, 0, 5], x[2, 1, 100], x[3, 0, 40] = float("inf"), float("nan"), float("-inf")
    for side, partner in ((False, {5: 69, 100: 36, 40: 104}), (True, {5: 4, 100: 101, 40: 41})):
        y = torch.empty((4, 2, DIM), dtype=torch.bfloat16, device="cuda")
        B.pa_rotate(x.cuda(), pos.cuda(), B.make_rotation(128, interleaved=side), y)
        ok()
        bad = ~torch.isfinite(y.cpu())
        assert sorted(map(tuple, bad.nonzero().tolist())) == sorted(
            [(1, 0, 5), (1, 0, partner[5]), (2, 1, 100), (2, 1, partner[100]), (3, 0, 40),
             (3, 0, partner[40])])


def test_rows_beyond_a_32_bit_offset():
    # token stride 2^28 elements: the last token lies 2^32 bytes and more behind the first
    n = 9
    try:
        room = torch.zeros(((n - 1) << 28) + 4 * DIM, dtype=torch.bfloat16, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("no room")
    x = room.as_strided((n, 2, DIM), (1 << 28, DIM, 1))
    g = torch.Generator().manual_seed(6)
    small, pos = randn(g, n, 2, DIM).cuda(), positions_of(g, n).cuda()
    x.copy_(small)
    rot = B.make_rotation(128)
    B.pa_rotate(x, pos, rot, x)
    B.pa_rotate(small, pos, rot, small)
    ok()
    assert torch.equal(bits(x), bits(small))


def test_another_stream_and_a_graph():
    g = torch.Generator().manual_seed(7)
    x, pos = randn(g, 64, 8, DIM).cuda(), positions_of(g, 64).cuda()
    rot, y, want = B.make_rotation(128), torch.empty_like(x), torch.empty_like(x)
    B.pa_rotate(x, pos, rot, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = B.prepare_rotate(x, pos, rot, y)
        call()
    ok()
    assert torch.equal(bits(y), bits(want))
    rot.turns[3] = 0  # a prepared call keeps the map that it was made with
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x2, pos2 = randn(g, 64, 8, DIM).cuda(), positions_of(g, 64, 99).cuda()
    x.copy_(x2)
    pos.copy_(pos2)
    graph.replay()
    B.pa_rotate(x2, pos2, B.make_rotation(128), want)
    ok()
    assert torch.equal(bits(y), bits(want))


# ---------------------------------------------------------------------------
# pa_rotate_and_cache
# ---------------------------------------------------------------------------

def empty_pool(blocks, hkv, fmt):
    if fmt == "bf16":
        return torch.full((blocks, hkv, BLOCK, DIM), 77.0, dtype=torch.bfloat16, device="cuda")
    return torch.full((blocks, hkv, TILE), 0xA5, dtype=torch.uint8, device="cuda")


def plain_write(k, v, slots, kc, vc, fmt):
    {"bf16": B.pa_reshape_and_cache, "int8": B.pa_reshape_and_cache_int8,
     "fp8": B.pa_reshape_and_cache_fp8}[fmt](k.contiguous(), v.contiguous(), slots, kc, vc)


APPENDS = [
    # tokens, query heads (0: none), KV heads, rotated dimensions, interleaved
    (1, 16, 8, 128, False),
    (4, 2, 1, 128, True),
    (19, 0, 8, 64, False),
    (33, 12, 4, 96, True),
    (50, 15, 5, 30, False),
    (7, 40, 2, 128, False),
    (130, 3, 3, 112, False),
]


@pytest.mark.parametrize("T,hq,hkv,r,side", APPENDS)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_a_steps_rows_into_the_cache(T, hq, hkv, r, side, fmt):
    g = torch.Generator().manual_seed(T * 31 + hq)
    mixed = randn(g, T, hq + 2 * hkv, DIM)
    mixed[T // 2, hq] = 0            # a key of zeros
    pos = positions_of(g, T)
    blocks = T // 4 + 3
    slots = torch.randperm(blocks * BLOCK, generator=g)[:T]
    if T > 3:
        slots[3] = -1                # its row stays out
    rot, (th, m) = B.make_rotation(r, interleaved=side), R.theta(r)
    d = mixed.cuda()
    q, k, v = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:]
    kc, vc = empty_pool(blocks, hkv, fmt), empty_pool(blocks, hkv, fmt)
    q_out = torch.full((T, hq, DIM), 3.0, dtype=torch.bfloat16, device="cuda") if hq else None
    B.pa_rotate_and_cache(k, v, pos.cuda(), slots.cuda(), rot, kc, vc, q=q if hq else None,
                          q_out=q_out, kv_format=KIND[fmt])
    ok()
    # values, and what no token wrote: the bytes of the plain write
    kp, vp = empty_pool(blocks, hkv, fmt), empty_pool(blocks, hkv, fmt)
    plain_write(k, v, slots.cuda(), kp, vp, fmt)
    ok()
    assert torch.equal(vc, vp) if fmt != "bf16" else torch.equal(bits(vc), bits(vp))
    written = slots[slots >= 0]
    rest = torch.ones(blocks * BLOCK, dtype=torch.bool)
    rest[written] = False
    ref, err = R.rotate(k.cpu(), pos[:, None], th, side, m)
    ref, err = ref[slots >= 0], err[slots >= 0]
    if fmt == "bf16":
        rows = kc.cpu().transpose(1, 2).reshape(blocks * BLOCK, hkv, DIM)
        assert (rows[rest] == 77).all()
        tol = R.held_bf16(ref, err)
        got = rows[written].double()
        # the same bits as the rows' own rotation
        same = torch.empty_like(k.contiguous())
        B.pa_rotate(k, pos.cuda(), rot, same)
        assert torch.equal(bits(rows[written]), bits(same.cpu()[slots >= 0]))
    else:
        raw = kc.cpu()
        codes = raw[..., :2048].unflatten(-1, (BLOCK, DIM)).transpose(1, 2).flatten(0, 1)
        scale = raw[..., 2048:].unflatten(-1, (BLOCK, 4)).transpose(1, 2).flatten(0, 1)
        assert (codes[rest] == 0xA5).all() and (scale[rest] == 0xA5).all()
        got = R.tiles_values(raw, fmt).transpose(1, 2).flatten(0, 1)[written]
        tol = R.held_codes(ref, err, fmt)
    assert ((got - ref).abs() <= tol).all()
    if hq:
        qr, qe = R.rotate(q.cpu(), pos[:, None], th, side, m)
        assert ((q_out.cpu().double() - qr).abs() <= R.held_bf16(qr, qe)).all()
        # in place in the fused rows
        before = d.clone()
        kc2, vc2 = empty_pool(blocks, hkv, fmt), empty_pool(blocks, hkv, fmt)
        B.pa_rotate_and_cache(k, v, pos.cuda(), slots.cuda(), rot, kc2, vc2, q=q, q_out=q,
                              kv_format=KIND[fmt])
        ok()
        assert torch.equal(bits(q.contiguous()), bits(q_out))
        assert torch.equal(bits(d[:, hq:].contiguous()), bits(before[:, hq:].contiguous()))
        assert torch.equal(kc2.view(torch.uint8), kc.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_a_slot_outside_the_pool_is_flagged(fmt):
    g = torch.Generator().manual_seed(9)
    for hq in (0, 1, 8, 9):
        hkv = 1 if hq in (0, 1) else hq
        d = randn(g, 3, hq + 2 * hkv, DIM).cuda()
        pos = torch.arange(3, dtype=torch.int32, device="cuda")
        slots = torch.tensor([5, 64, 7], device="cuda")
        kc, vc = empty_pool(4, hkv, fmt), empty_pool(4, hkv, fmt)
        q = d[:, :hq] if hq else None
        q_out = torch.zeros((3, hq, DIM), dtype=torch.bfloat16, device="cuda") if hq else None
        rot = B.make_rotation(128)
        B.pa_rotate_and_cache(d[:, hq:hq + hkv], d[:, hq + hkv:], pos, slots, rot, kc, vc, q=q,
                              q_out=q_out, kv_format=KIND[fmt])
        torch.cuda.synchronize()
        assert B.pa_debug_read_error() == B.PA_DEVERR_SLOT_RANGE
        want, _ = empty_pool(4, hkv, fmt), None
        wv = empty_pool(4, hkv, fmt)
        B.pa_rotate_and_cache(d[:, hq:hq + hkv], d[:, hq + hkv:], pos,
                              torch.tensor([5, -1, 7], device="cuda"), rot, want, wv,
                              kv_format=KIND[fmt])
        ok()
        assert torch.equal(kc.view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(vc.view(torch.uint8), wv.view(torch.uint8))
        if hq:  # the token's query is rotated all the same
            qr, qe = R.rotate(q.cpu(), pos.cpu()[:, None], R.theta(128)[0], False)
            assert ((q_out.cpu().double() - qr).abs() <= R.held_bf16(qr, qe)).all()


# ---------------------------------------------------------------------------
# pa_rotate_cached
# ---------------------------------------------------------------------------

def filled_pool(g, blocks, hkv, fmt):
    """A pool of random rows, its 8-bit form written by the library's own write."""
    k = randn(g, blocks * BLOCK, hkv, DIM).cuda()
    kc, vc = empty_pool(blocks, hkv, fmt), empty_pool(blocks, hkv, fmt)
    plain_write(k, k, torch.arange(blocks * BLOCK, device="cuda"), kc, vc, fmt)
    ok()
    return kc


def tables_of(g, lens, width=None):
    per = [(n + BLOCK - 1) // BLOCK for n in lens]
    blocks = sum(per) + 3
    ids = torch.randperm(blocks, generator=g).to(torch.int32)
    t = torch.full((len(lens), width or max(max(per), 1)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(per):
        t[s, :n] = ids[at:at + n]
        at += n
    return t, blocks


def check_moved(before, after, tables, lens, by, th, side, fmt):
    """by [S][hkv][positions]: every key's turn."""
    def whole(p):
        return p.cpu().double() if fmt == "bf16" else R.tiles_values(p.cpu(), fmt)
    old, new = whole(before), whole(after)
    raw_old, raw_new = before.cpu(), after.cpu()
    turned = torch.zeros(old.shape[:3], dtype=torch.bool)
    for s, c in enumerate(lens):
        for h in range(old.shape[1]):
            i = torch.arange(c)
            b = by[s][h][:c]
            i, b = i[b != 0], b[b != 0]
            ids = tables[s, i // BLOCK].long()
            turned[ids, h, i % BLOCK] = True
            ref, err = R.rotate(old[ids, h, i % BLOCK], b, th, side)
            if fmt == "bf16":
                tol = R.held_bf16(ref, err)
            else:
                # the value itself enters as a code times its scale, rounded to fp32
                tol = R.held_codes(ref, err + 2.0 ** -23 * ref.abs(), fmt)
            assert ((new[ids, h, i % BLOCK] - ref).abs() <= tol).all(), (s, h)
    if fmt == "bf16":
        assert torch.equal(bits(raw_old)[~turned], bits(raw_new)[~turned])
    else:
        codes = [x[..., :2048].unflatten(-1, (BLOCK, DIM))[~turned] for x in (raw_old, raw_new)]
        scale = [x[..., 2048:].unflatten(-1, (BLOCK, 4))[~turned] for x in (raw_old, raw_new)]
        assert torch.equal(*codes) and torch.equal(*scale)


MOVES = [
    ([1], 1, 128, False), ([0, 17, 16, 15], 2, 128, True), ([300, 33, 0, 1], 3, 64, False),
    ([77, 200], 8, 30, False), ([1000], 1, 96, True), ([64, 64], 2, 112, False),
]


@pytest.mark.parametrize("lens,hkv,r,side", MOVES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_cached_keys_by_a_shift(lens, hkv, r, side, fmt):
    g = torch.Generator().manual_seed(len(lens) * 100 + r)
    tables, blocks = tables_of(g, lens, width=80)
    pool = filled_pool(g, blocks, hkv, fmt)
    before = pool.clone()
    shifts = torch.randint(-5000, 100, (len(lens),), generator=g, dtype=torch.int32)
    shifts[0] = 0 if len(lens) > 1 else -7
    first = 5
    rot, (th, _) = B.make_rotation(r, interleaved=side), R.theta(r)
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), rot,
                       shifts=shifts.cuda(), first=first, kv_format=KIND[fmt])
    ok()
    by = [[torch.where(torch.arange(n) >= first, shifts[s].long(), 0)] * hkv
          for s, n in enumerate(lens)]
    check_moved(before, pool, tables, lens, by, th, side, fmt)


@pytest.mark.parametrize("lens,hkv,r,side", MOVES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_cached_keys_by_what_was_kept(lens, hkv, r, side, fmt):
    g = torch.Generator().manual_seed(len(lens) * 77 + r)
    tables, blocks = tables_of(g, lens)
    pool = filled_pool(g, blocks, hkv, fmt)
    before = pool.clone()
    n = max(3, max(lens) - 4)   # the last positions of the longest have no entry: they stay
    kept = torch.arange(n) + (torch.rand((len(lens), hkv, n), generator=g) < 0.3).long().cumsum(-1)
    kept[:, :, :2] = torch.arange(2)
    kept[torch.rand(kept.shape, generator=g) < 0.05] = -1
    rot, (th, _) = B.make_rotation(r, interleaved=side), R.theta(r)
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), rot,
                       kept=kept.to(torch.int32).cuda(), kv_format=KIND[fmt])
    ok()
    by = []
    for s, c in enumerate(lens):
        row = torch.zeros(hkv, max(c, n), dtype=torch.int64)
        row[:, :n] = torch.where(kept[s] >= 0, torch.arange(n) - kept[s], 0)
        by.append(row)
    check_moved(before, pool, tables, lens, by, th, side, fmt)


def test_int8_codes_of_ties_extremes_and_nans():
    # amax 127, so that a value is its own code: integers, halves between (to even), tiny ones
    x = torch.zeros(3, 1, 128)
    x[0, 0, :127] = torch.arange(127).float() - 63.5
    x[1, 0, :127] = torch.arange(-127, 0).float()
    x[2, 0, :12] = torch.tensor([0.5, 1.5, -0.5, -2.5, 1e-30, -1e-38, 126.5, -126.5, 3.25, -0.0,
                                 float("nan"), 7.0])
    x[:, 0, 127] = 127.0
    x = x.to(torch.bfloat16).cuda()
    kc, vc = empty_pool(1, 1, "int8"), empty_pool(1, 1, "int8")
    slots = torch.arange(3, dtype=torch.int64, device="cuda")
    plain_write(x, x, slots, kc, vc, "int8")
    ok()
    got = kc[0, 0, :384].view(torch.int8).view(3, 128).cpu()
    want = x[:, 0].float().cpu().round()
    want = torch.where(want.isnan(), torch.tensor(-127.0), want).to(torch.int8)
    assert torch.equal(got, want)
    assert torch.equal(vc, kc)
    assert (kc[0, 0, 2048:2060].view(torch.float32).cpu() == 1.0).all()


def test_every_int8_code_passes_a_turn_by_nothing():
    # an angle of zero: read as values, turned, written as codes again
    codes = torch.empty(16, 128, dtype=torch.int8)
    codes[0::2] = torch.arange(-127, 1).to(torch.int8)
    codes[1::2] = torch.arange(0, 128).to(torch.int8)
    pool = torch.zeros(1, 1, TILE, dtype=torch.uint8)
    pool[0, 0, :2048] = codes.view(torch.uint8).flatten()
    scales = 2.0 ** (torch.arange(16) * 5.0 - 40) * (1 + torch.arange(16) / 37)
    pool[0, 0, 2048:] = scales.float().view(torch.uint8)
    pool = pool.cuda()
    before = pool.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    B.pa_rotate_cached(pool, torch.zeros(1, 1, **i32), torch.tensor([16], **i32),
                       B.make_rotation_from([0.0] * 64), shifts=torch.tensor([3], **i32),
                       kv_format=B.PA_KV_INT8)
    ok()
    assert torch.equal(pool[0, 0, :2048], before[0, 0, :2048])
    a, b = (x[0, 0, 2048:].view(torch.float32).cpu() for x in (pool, before))
    assert ((a - b).abs() <= 2.0 ** -22 * b).all()   # code times scale, amax over 127: two roundings


def test_moved_keys_leave_out_the_magnitude():
    g = torch.Generator().manual_seed(3)
    tables, blocks = tables_of(g, [40])
    pool = filled_pool(g, blocks, 2, "bf16")
    before = pool.clone()
    kw = dict(base=1e6, scaling="ramp", factor=4.0, original_len=32768, high=32.0)
    B.pa_rotate_cached(pool, tables.cuda(), torch.tensor([40], dtype=torch.int32).cuda(),
                       B.make_rotation(128, **kw),
                       shifts=torch.tensor([-9], dtype=torch.int32).cuda())
    ok()
    by = [[torch.full((40,), -9)] * 2]
    check_moved(before, pool, tables, [40], by, R.theta(128, **kw)[0], False, "bf16")


def test_bad_blocks_and_contexts_of_moved_keys_are_flagged():
    g = torch.Generator().manual_seed(3)
    tables, blocks = tables_of(g, [40, 64])
    pool = filled_pool(g, blocks, 2, "bf16")
    before = pool.clone()
    rot, shifts = B.make_rotation(128), torch.tensor([-9, 0], dtype=torch.int32).cuda()
    lens = torch.tensor([40, 64], dtype=torch.int32).cuda()
    bad = tables.clone()
    bad[0, 1] = blocks
    B.pa_rotate_cached(pool, bad.cuda(), lens, rot, shifts=shifts)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_BLOCK_RANGE
    keep = torch.arange(40)
    by = [[torch.where((keep < 16) | (keep >= 32), -9, 0)] * 2, [torch.zeros(64).long()] * 2]
    check_moved(before, pool, tables, [40, 64], by, R.theta(128)[0], False, "bf16")
    lens[1] = 65
    B.pa_rotate_cached(pool, tables.cuda(), lens, rot, shifts=shifts * 0)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_CONTEXT_RANGE


def test_many_sequences_turn_the_same_as_one_by_one():
    g = torch.Generator().manual_seed(12)
    lens = [int(x) for x in torch.randint(0, 90, (700,), generator=g)]
    tables, blocks = tables_of(g, lens)
    pool = filled_pool(g, blocks, 1, "bf16")
    other = pool.clone()
    shifts = torch.randint(-50, 50, (700,), generator=g, dtype=torch.int32).cuda()
    rot, lens_d = B.make_rotation(128), torch.tensor(lens, dtype=torch.int32).cuda()
    B.pa_rotate_cached(pool, tables.cuda(), lens_d, rot, shifts=shifts)
    for s in range(0, 700, 100):
        B.pa_rotate_cached(other, tables[s:s + 100].cuda(), lens_d[s:s + 100].contiguous(), rot,
                           shifts=shifts[s:s + 100].contiguous())
    ok()
    assert torch.equal(bits(pool), bits(other))


# ---------------------------------------------------------------------------
# a run of them
# ---------------------------------------------------------------------------

def test_a_cache_is_filled_read_shrunk_and_moved():
    """Keys rotated into the cache, attention over them, an eviction by the
    weights that they drew, the kept keys turned to their new positions: they are
    then what a cache filled at those positions holds."""
    g = torch.Generator().manual_seed(21)
    lens, hq, hkv, budget = [90, 40, 161], 4, 2, 64
    tables, blocks = tables_of(g, lens)
    T = sum(lens)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens))
    pos = torch.cat([torch.arange(n) for n in lens])
    slots = (tables[seq, pos // BLOCK].long() * BLOCK + pos % BLOCK).cuda()
    mixed = randn(g, T, hq + 2 * hkv, DIM).cuda()
    q, k, v = mixed[:, :hq], mixed[:, hq:hq + hkv], mixed[:, hq + hkv:]
    rot, (th, _) = B.make_rotation(128), R.theta(128)
    kc, vc = empty_pool(blocks, hkv, "bf16"), empty_pool(blocks, hkv, "bf16")
    q_out = torch.empty((T, hq, DIM), dtype=torch.bfloat16, device="cuda")
    lens_d, tab_d = torch.tensor(lens, dtype=torch.int32).cuda(), tables.cuda()
    B.pa_rotate_and_cache(k, v, pos.int().cuda(), slots, rot, kc, vc, q=q, q_out=q_out)
    last = torch.tensor(np.cumsum(lens) - 1).cuda()
    qd = q_out[last].contiguous()
    out = torch.empty_like(qd)
    lse = torch.empty((3, hq), dtype=torch.float32, device="cuda")
    sh = B.shape_of(qd, kc, tab_d)
    ws = B.workspace(B.pa_decode_workspace_size(sh), "cuda")
    scale = 1 / math.sqrt(DIM)
    B.pa_decode(qd, kc, vc, tab_d, lens_d, scale, out, lse, workspace=ws)
    ok()
    # attention with keys and queries turned in 64 bits
    for s, n in enumerate(lens):
        rows = (seq == s).nonzero()[:, 0]
        kr, ke = R.rotate(k.cpu()[rows], pos[rows][:, None], th, False)
        qr, qe = R.rotate(q.cpu()[rows[-1:]], pos[rows[-1:]][:, None], th, False)
        for h in range(hq):
            kk, qq, vv = kr[:, h // 2], qr[0, h], v.cpu()[rows][:, h // 2].double()
            z = scale * (kk @ qq)
            p = torch.softmax(z, 0)
            # scores: both factors rounded to bf16, 128 terms summed in fp32; weights by
            # twice that, the output by the weights' error and its own rounding
            tk, tq = R.held_bf16(kr, ke)[:, h // 2], R.held_bf16(qr, qe)[0, h]
            dz = scale * (tk @ qq.abs() + kk.abs() @ tq + tk @ tq) + 2.0 ** -15 * z.abs().max()
            e = 2 * dz.max()
            tol = (math.exp(e) - 1) * (p @ vv.abs()) + 2 * R.UBF * (p @ vv.abs())
            assert ((out[s, h].cpu().double() - p @ vv).abs() <= tol).all()
            assert abs(float(lse[s, h]) - float(torch.logsumexp(z, 0))) <= float(dz.max()) + 1e-5
    weights = torch.zeros((3, hkv, tables.shape[1] * BLOCK), dtype=torch.float32, device="cuda")
    B.pa_accumulate_weights(qd, kc, lse, tab_d, lens_d, scale, weights, accumulate=False)
    kept = torch.empty((3, hkv, budget), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((3,), dtype=torch.int32, device="cuda")
    B.pa_evict(kc, vc, tab_d, lens_d, weights, torch.full((3,), budget, dtype=torch.int32).cuda(), 4,
               16, kept, new_lens)
    B.pa_rotate_cached(kc, tab_d, new_lens, rot, kept=kept)
    ok()
    start = np.concatenate([[0], np.cumsum(lens)])
    for s, n in enumerate(new_lens.tolist()):
        assert n == min(lens[s], budget)
        i = torch.arange(n)
        ids = tables[s, i // BLOCK].long()
        for h in range(hkv):
            old = kept[s, h, :n].cpu().long()
            rows = int(start[s]) + old
            ref, err = R.rotate(k.cpu()[rows, h], i, th, False)
            # rounded to bf16 at its first position, turned on (a pair's error becomes
            # at most the sum of both), rounded again
            first, ferr = R.rotate(k.cpu()[rows, h], old, th, False)
            f = R.held_bf16(first, ferr)
            pair = f.clone()
            pair[:, :64] = pair[:, 64:] = f[:, :64] + f[:, 64:]
            got = kc.cpu()[ids, h, i % BLOCK].double()
            assert ((got - ref).abs() <= R.held_bf16(ref, 2 * err + pair)).all()
