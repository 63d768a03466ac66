"""Differential attention over the paged cache on the GPU, against a plain
64-bit form."""
import math

import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from tests import diff_ref as R
from tests import rotate_ref

pytestmark = pytest.mark.gpu

DIM, BLOCK = 128, 16
SCALE = 1 / math.sqrt(DIM)


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


class Batch:
    """A batch in a shuffled pool: contexts `lens`, windows `qs` (None: one query
    per sequence), cached rows past a context and unused blocks NaN."""

    def __init__(self, seed, lens, qs, hkv, G, width=0, heavy=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.qs, self.hkv, self.G, self.hq = lens, qs, hkv, G, hkv * G
        per = [(n + BLOCK - 1) // BLOCK for n in lens]
        blocks = sum(per) + 2
        ids = torch.randperm(blocks, generator=g).to(torch.int32)
        self.tables = torch.full((len(lens), max(width, max(per), 1)), -1, dtype=torch.int32)
        self.kc = torch.full((blocks, hkv, BLOCK, DIM), float("nan"), dtype=torch.bfloat16)
        self.vc = self.kc.clone()
        at = 0
        for s, n in enumerate(lens):
            mine = ids[at:at + per[s]]
            self.tables[s, :per[s]] = mine
            at += per[s]
            for pool, gain in ((self.kc, heavy), (self.vc, 1.0)):
                x = randn(g, n, hkv, DIM)
                if gain != 1.0 and n:
                    x[torch.rand((n,), generator=g) < 0.05] *= gain
                for b in range(per[s]):
                    part = x[b * BLOCK:(b + 1) * BLOCK]
                    pool[int(mine[b]), :, :part.shape[0]] = part.transpose(0, 1)
        rows = [1] * len(lens) if qs is None else qs
        self.cu = torch.tensor([0] + rows, dtype=torch.int64).cumsum(0).to(torch.int32)
        self.T = int(self.cu[-1])
        self.q = randn(g, self.T, self.hq, DIM)
        self.lambdas = torch.rand((self.hq // 2,), generator=g) * 1.2 - 0.2
        self.weight = 1 + 0.2 * torch.randn((2 * DIM,), generator=g)
        self.max_q = max(rows) if rows else 1

    def cuda(self):
        self.d = {n: getattr(self, n).cuda() for n in
                  ("q", "kc", "vc", "tables", "lambdas", "weight", "cu")}
        self.d["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self

    def call(self, norm=True, eps=1e-5, gain=0.8, causal=True, with_lse=True, max_q=None,
             spare=0, ws_fill=None, workspace=None):
        d = self.d
        out = torch.full((self.T + spare, self.hq // 2, 2 * DIM), 3.0, dtype=torch.bfloat16,
                         device="cuda")
        lse = torch.full((self.T + spare, self.hq), 5.0, device="cuda") if with_lse else None
        sh = B.shape_of(d["q"], d["kc"], d["tables"])
        n = max_q or self.max_q
        ws = workspace
        if ws is None:
            ws = B.workspace(B.pa_decode_diff_workspace_size(sh, self.T, n), "cuda")
            if ws_fill is not None:
                ws.fill_(ws_fill)
        B.pa_decode_diff(d["q"], d["kc"], d["vc"], d["tables"], d["lens"], SCALE, d["lambdas"],
                         out[:self.T], None if lse is None else lse[:self.T],
                         cu_seqlens_q=None if self.qs is None else d["cu"], max_q_len=n,
                         causal=causal, norm_weight=d["weight"] if norm else None, norm_eps=eps,
                         out_scale=gain, workspace=ws)
        return out, lse

    def check(self, out, lse, norm=True, eps=1e-5, gain=0.8, causal=True):
        ref, rl, tol, ltol = R.attend(self.q, self.kc, self.vc, self.tables, self.lens, self.cu,
                                      SCALE, self.lambdas, self.weight if norm else None, eps, gain,
                                      causal)
        got = out[:self.T].cpu().double()
        assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())
        # the bounds say little of a difference that is small beside its maps: all in
        # all the error is a few roundings of random sign
        if ref.norm() > 0:
            assert float((got - ref).norm() / ref.norm()) < 1e-2
        if lse is not None:
            gl = lse[:self.T].cpu().double()
            empty = torch.isinf(rl)
            assert torch.equal(gl[empty], rl[empty])
            assert ((gl - rl).abs() <= ltol)[~empty].all()


DECODE = [
    # contexts, KV heads, group
    ([1], 2, 1), ([16], 2, 2), ([0, 17, 1, 15, 33, 0], 2, 1), ([300, 5, 129], 8, 2),
    ([40, 64], 4, 3), ([65, 31], 2, 5), ([70], 6, 4), ([257, 9], 2, 8), ([33, 100], 4, 7),
    # few segments in many pieces
    ([5000], 2, 1), ([3000, 40], 4, 2), ([2600], 2, 8),
]


@pytest.mark.parametrize("lens,hkv,G", DECODE)
@pytest.mark.parametrize("norm", [True, False])
def test_one_query_per_sequence(lens, hkv, G, norm):
    b = Batch(len(lens) * 100 + lens[0] + G, lens, None, hkv, G, heavy=4.0).cuda()
    out, lse = b.call(norm=norm, spare=2, ws_fill=0xFF)
    ok()
    b.check(out, lse, norm=norm)
    assert (out[b.T:] == 3).all() and (lse[b.T:] == 5).all()
    again, _ = b.call(norm=norm, with_lse=False, ws_fill=0x11)
    ok()
    assert torch.equal(again[:b.T].view(torch.int16), out[:b.T].view(torch.int16))
    for s, c in enumerate(lens):
        if c == 0:
            assert (out[s] == 0).all() and (lse[s] == -math.inf).all()


WINDOWS = [
    # contexts, windows, KV heads, group
    ([1], [1], 2, 1), ([20, 16, 40], [5, 16, 0], 2, 2), ([64, 65, 7], [1, 33, 7], 4, 1),
    ([100, 30], [9, 30], 2, 3), ([50], [50], 2, 8), ([129, 200, 17], [4, 8, 17], 2, 5),
    ([900, 33], [12, 3], 4, 2), ([80, 0, 90], [20, 0, 31], 6, 4), ([210], [70], 2, 6),
]


@pytest.mark.parametrize("lens,hkv,G", DECODE)
def test_one_query_per_sequence_under_a_wide_table(lens, hkv, G):
    # the table's width chooses how the batch is cut
    b = Batch(len(lens) * 100 + lens[0] + G, lens, None, hkv, G, width=400, heavy=4.0).cuda()
    out, lse = b.call(ws_fill=0xFF)
    ok()
    b.check(out, lse)


@pytest.mark.parametrize("lens,qs,hkv,G", WINDOWS)
def test_windows_under_a_wide_table(lens, qs, hkv, G):
    b = Batch(sum(lens) + hkv, lens, qs, hkv, G, width=400).cuda()
    out, lse = b.call(ws_fill=0xFF)
    ok()
    b.check(out, lse)


@pytest.mark.parametrize("lens,hkv,G", [
    ([1000, 3, 1024, 0, 700] + [16 * i + 5 for i in range(45)], 4, 2),   # a CTA to 100 segments
    ([500] * 38, 8, 1), ([448, 1, 0, 2], 2, 8), ([449], 2, 3), ([5, 80, 79, 81], 4, 1),
])
def test_segments_of_one_cta(lens, hkv, G):
    b = Batch(51 + G, lens, None, hkv, G, heavy=3.0).cuda()
    out, lse = b.call(ws_fill=0x7f)
    ok()
    b.check(out, lse)
    again, _ = b.call(norm=True, with_lse=False)
    ok()
    assert torch.equal(again[:b.T].view(torch.int16), out[:b.T].view(torch.int16))


@pytest.mark.parametrize("lens,qs,hkv,G", WINDOWS)
@pytest.mark.parametrize("causal", [True, False])
def test_windows(lens, qs, hkv, G, causal):
    b = Batch(sum(lens) + G, lens, qs, hkv, G, heavy=4.0).cuda()
    out, lse = b.call(causal=causal, spare=3)
    ok()
    b.check(out, lse, causal=causal)
    assert (out[b.T:] == 3).all() and (lse[b.T:] == 5).all()
    # a wider bound of the windows is the same problem
    again, _ = b.call(causal=causal, max_q=b.max_q + 9)
    ok()
    b.check(again, None, causal=causal)


LONG = [
    # windows of several tiles of 256 rows, and rows that fill none
    ([128], [128], 2, 1), ([300, 129], [257, 64], 2, 2), ([1000, 70, 515], [130, 70, 1], 4, 2),
    ([640], [512], 2, 4), ([200, 90], [90, 33], 2, 3), ([333], [200], 2, 8), ([140, 3], [20, 3], 2, 7),
    # more heads to a KV head than a warp tile holds
    ([40, 0, 200], [5, 0, 1], 2, 16), ([77], [30], 2, 24), ([100, 260], [2, 3], 2, 128),
    # few segments in many pieces
    ([4000], [64], 2, 1), ([3000, 200], [70, 100], 2, 2),
]


@pytest.mark.parametrize("lens,qs,hkv,G", LONG)
@pytest.mark.parametrize("causal,norm", [(True, True), (False, False)])
def test_long_windows(lens, qs, hkv, G, causal, norm):
    b = Batch(sum(lens) + G, lens, qs, hkv, G, heavy=4.0).cuda()
    out, lse = b.call(causal=causal, norm=norm, spare=3, ws_fill=0xFF)
    ok()
    b.check(out, lse, causal=causal, norm=norm)
    assert (out[b.T:] == 3).all() and (lse[b.T:] == 5).all()
    again, _ = b.call(causal=causal, norm=norm, with_lse=False, ws_fill=0x11)
    ok()
    assert torch.equal(again[:b.T].view(torch.int16), out[:b.T].view(torch.int16))


@pytest.mark.parametrize("lens,G", [([33, 0, 1], 9), ([300], 32), ([2000, 17], 16)])
def test_single_queries_of_many_heads(lens, G):
    b = Batch(sum(lens) + G, lens, None, 2, G).cuda()
    out, lse = b.call()
    ok()
    b.check(out, lse)
    for s, c in enumerate(lens):
        if c == 0:
            assert (out[s] == 0).all() and (lse[s] == -math.inf).all()


def test_a_hidden_key_of_a_long_window_never_reaches_a_query():
    lens, qs = [700, 200], [300, 150]
    b = Batch(3, lens, qs, 2, 2)
    clean = b.kc.clone(), b.vc.clone()
    # (one head's values alone, in either sequence: the tile's halves hold one each)
    for s, at, h, what in ((0, 600, 0, float("nan")), (0, 650, 1, float("inf")),
                           (1, 120, 1, float("-inf"))):
        blk = int(b.tables[s, at // BLOCK])
        b.kc[blk, :, at % BLOCK, 3::7] = what
        b.vc[blk, h, at % BLOCK, 1::5] = what
    b.cuda()
    out, lse = b.call()
    ok()
    ref, rl, tol, ltol = R.attend(b.q, *clean, b.tables, lens, b.cu, SCALE, b.lambdas, b.weight,
                                  1e-5, 0.8)
    got, gl = out.cpu().double(), lse.cpu().double()
    fine = torch.zeros(b.T, dtype=torch.bool)
    fine[0:200] = True               # positions 400 .. 599
    fine[300:370] = True             # positions 50 .. 119
    assert ((got - ref).abs() <= tol)[fine].all()
    assert ((gl - rl).abs() <= ltol)[fine].all()
    assert not torch.isfinite(got[~fine]).all(-1).any()


def test_values_that_are_infinite_where_they_are_seen():
    # finite scores: the queries from the key on get the infinity, the others none
    for lens, qs in (([700], [300]), ([60], [20])):
        b = Batch(4, lens, qs, 2, 1)
        at = lens[0] - 10
        b.vc[int(b.tables[0, at // BLOCK]), 1, at % BLOCK, 7] = float("inf")
        b.cuda()
        out, _ = b.call(norm=False)
        ok()
        bad = ~torch.isfinite(out[:b.T, 0].cpu())
        want = torch.zeros_like(bad)
        want[qs[0] - 10:, DIM + 7] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("G", [1, 2, 8])
@pytest.mark.parametrize("ctx", [600, 1337, 20000])
def test_infinite_values_in_every_part_of_a_long_window(G, ctx):
    # one to five query tiles of a window of 600: an infinity in a tile's own rows reaches
    # the queries from its own on, one in an earlier tile's all of the tile
    b = Batch(21, [ctx], [600], 2, G)
    spots = ((ctx - 600 + 40, 0, 7), (ctx - 600 + 300, 1, 9), (ctx - 600 + 555, 0, 100))
    for at, h, dim in spots:
        b.vc[int(b.tables[0, at // BLOCK]), h, at % BLOCK, dim] = float("inf")
    b.cuda()
    out, lse = b.call(norm=False)
    ok()
    bad = ~torch.isfinite(out[:b.T].cpu())
    want = torch.zeros_like(bad)
    for at, h, dim in spots:
        want[at - ctx + 600:, :, h * DIM + dim] = True
    assert torch.equal(bad, want)
    for at, h, dim in spots:
        b.vc[int(b.tables[0, at // BLOCK]), h, at % BLOCK, dim] = 0.0
    ref, rl, tol, ltol = R.attend(b.q, b.kc, b.vc, b.tables, b.lens, b.cu, SCALE, b.lambdas, None,
                                  1e-5, 0.8)
    got = out[:b.T].cpu().double()
    assert ((got - ref).abs() <= tol)[~want].all()
    assert ((lse[:b.T].cpu().double() - rl).abs() <= ltol).all()


@pytest.mark.parametrize("lens,hkv,G", [
    ([5000, 0, 17, 0, 500], 2, 2),                                   # many pieces, by segment
    ([0, 0, 0, 4000], 4, 1),
    ([16, 16, 3000], 2, 8),                                          # whole segments among them
    ([0] + [7 + 13 * i % 90 if i % 3 else 0 for i in range(330)], 2, 1),   # mostly by boundary
    ([9000] + [5] * 300, 2, 2),                                      # one of many pieces
    ([40 * i for i in range(60)] + [0], 2, 5),
])
@pytest.mark.parametrize("fill", [0, 0x7f, 0xff])
def test_whatever_the_workspace_held(lens, hkv, G, fill):
    # descriptors and partials of an earlier call mean nothing; empty contexts between others
    b = Batch(31, lens, None, hkv, G).cuda()
    out, lse = b.call(ws_fill=fill)
    ok()
    b.check(out, lse)


@pytest.mark.parametrize("lens,qs,hkv,G", [
    ([12900 + 77 * i for i in range(8)], None, 8, 1),          # few segments, many pieces
    ([0, 30000, 5, 51000, 16, 0, 25000], None, 8, 2),          # empty and whole ones among them
    ([(997 * i) % 4100 for i in range(100)], None, 8, 1),      # ragged
    ([(997 * i) % 4100 + 4 for i in range(64)], [i % 4 for i in range(64)], 8, 2),
    ([98000, 100], [2, 1], 8, 3),
])
def test_large_batches(lens, qs, hkv, G):
    # thirty tiles of 16 keys of a pair and more for each of the workers
    b = Batch(41 + G, lens, qs, hkv, G, heavy=2.0).cuda()
    out, lse = b.call(ws_fill=0x7f)
    ok()
    b.check(out, lse)
    for fill in (0, 0xff):
        again, la = b.call(ws_fill=fill)
        ok()
        assert torch.equal(again[:b.T].view(torch.int16), out[:b.T].view(torch.int16))
        assert torch.equal(la[:b.T].view(torch.int32), lse[:b.T].view(torch.int32))


@pytest.mark.parametrize("lens,qs,T,max_q", [
    ([5000, 64], [3, 1], 20, 16),     # room for more windows than there are
    ([5000, 700], [16, 0], 16, 16),
])
def test_a_padded_batch_of_few_windows(lens, qs, T, max_q):
    b = Batch(32, lens, qs, 2, 1).cuda()
    d = b.d
    d["q"] = torch.cat([d["q"], torch.full((T - b.T, b.hq, DIM), float("nan"), dtype=torch.bfloat16,
                                           device="cuda")])
    out = torch.full((T, b.hq // 2, 2 * DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, b.hq), 5.0, device="cuda")
    sh = B.shape_of(d["q"], d["kc"], d["tables"])
    ws = B.workspace(B.pa_decode_diff_workspace_size(sh, T, max_q), "cuda")
    ws.fill_(0x11)
    B.pa_decode_diff(d["q"], d["kc"], d["vc"], d["tables"], d["lens"], SCALE, d["lambdas"], out, lse,
                     cu_seqlens_q=d["cu"], max_q_len=max_q, norm_weight=d["weight"], out_scale=0.8,
                     workspace=ws)
    ok()
    b.check(out, lse)
    assert (out[b.T:] == 3.0).all() and (lse[b.T:] == 5.0).all()


def test_short_and_long_windows_in_one_call():
    lens, qs = [900, 40, 333, 64], [200, 5, 100, 1]
    b = Batch(8, lens, qs, 4, 2).cuda()
    out, lse = b.call()
    ok()
    b.check(out, lse)


@pytest.mark.parametrize("lens,qs,T,max_q,G", [
    ([90, 40], [5, 3], 11, 5, 2),          # short windows
    ([300, 200], [64, 20], 128, 64, 1),    # as many rows as two windows of 64 would hold
    ([300, 200, 50], [70, 0, 2], 90, 70, 2),
])
def test_rows_behind_the_last_sequence_stay(lens, qs, T, max_q, G):
    b = Batch(14, lens, qs, 2, G).cuda()
    g = torch.Generator().manual_seed(1)
    more = T - b.T
    d = b.d
    d["q"] = torch.cat([d["q"], torch.full((more, b.hq, DIM), float("nan"), dtype=torch.bfloat16,
                                           device="cuda")])
    out = torch.full((T, b.hq // 2, 2 * DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, b.hq), 5.0, device="cuda")
    sh = B.shape_of(d["q"], d["kc"], d["tables"])
    ws = B.workspace(B.pa_decode_diff_workspace_size(sh, T, max_q), "cuda")
    B.pa_decode_diff(d["q"], d["kc"], d["vc"], d["tables"], d["lens"], SCALE, d["lambdas"], out, lse,
                     cu_seqlens_q=d["cu"], max_q_len=max_q, norm_weight=d["weight"], out_scale=0.8,
                     workspace=ws)
    ok()
    b.check(out, lse)
    assert (out[b.T:] == 3).all() and (lse[b.T:] == 5).all()


@pytest.mark.parametrize("lens,qs,G", [([5, 40], [9, 3], 2), ([20, 300], [90, 70], 2)])
def test_more_queries_than_keys_without_a_causal_mask(lens, qs, G):
    b = Batch(15, lens, qs, 2, G).cuda()
    out, lse = b.call(causal=False)
    ok()
    b.check(out, lse, causal=False)


def test_a_small_or_missing_workspace_is_refused():
    for qs, G in ((None, 2), ([3, 5], 2), ([40, 64], 2)):
        b = Batch(16, [90, 64], qs, 2, G).cuda()
        sh = B.shape_of(b.d["q"], b.d["kc"], b.d["tables"])
        need = B.pa_decode_diff_workspace_size(sh, b.T, b.max_q)
        assert need > 0
        for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
                   torch.empty(need + 256, dtype=torch.uint8, device="cuda")[8:]):
            with pytest.raises(B.PAError) as e:
                b.call(workspace=ws)
            assert e.value.status == B.PA_ERR_WORKSPACE


def test_two_graphs_that_share_a_workspace():
    a, c = Batch(51, [600, 40], None, 4, 2).cuda(), Batch(52, [300, 280], [100, 90], 4, 2).cuda()
    sizes, graphs = [], []
    for b in (a, c):
        sh = B.shape_of(b.d["q"], b.d["kc"], b.d["tables"])
        sizes.append(B.pa_decode_diff_workspace_size(sh, b.T, b.max_q))
    ws = B.workspace(max(sizes), "cuda")
    want = [b.call()[0].clone() for b in (a, c)]
    ok()
    outs = []
    for b in (a, c):
        d = b.d
        out = torch.zeros((b.T, b.hq // 2, 2 * DIM), dtype=torch.bfloat16, device="cuda")
        call = B.prepare_decode_diff(d["q"], d["kc"], d["vc"], d["tables"], d["lens"], SCALE,
                                     d["lambdas"], out,
                                     cu_seqlens_q=None if b.qs is None else d["cu"],
                                     max_q_len=b.max_q, norm_weight=d["weight"], out_scale=0.8,
                                     workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        for out in outs:
            out.zero_()
        for graph in graphs:
            graph.replay()
        ok()
        for out, w in zip(outs, want):
            assert torch.equal(out.view(torch.int16), w.view(torch.int16))


def test_a_pool_beyond_32_bit_offsets():
    # the sequences' blocks lie more than 2^32 bytes into either array
    far = (1 << 32) // (2 * BLOCK * DIM * 2) + 5
    for qs in (None, [40, 70]):
        b = Batch(61, [100, 90], qs, 2, 2)
        try:
            big = [torch.empty((far + b.kc.shape[0], 2, BLOCK, DIM), dtype=torch.bfloat16,
                               device="cuda") for _ in range(2)]
        except torch.cuda.OutOfMemoryError:
            pytest.skip("no room")
        b.cuda()
        big[0][far:], big[1][far:] = b.d["kc"], b.d["vc"]
        want, _ = b.call()
        b.d["kc"], b.d["vc"] = big
        b.d["tables"] = b.d["tables"] + far
        out, _ = b.call()
        ok()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        # the same keys turned there
        rot, shifts = B.make_rotation(128), torch.tensor([-7, 9], dtype=torch.int32).cuda()
        B.pa_rotate_cached(big[0], b.d["tables"], b.d["lens"], rot, shifts=shifts)
        near = b.kc.cuda()
        B.pa_rotate_cached(near, b.tables.cuda(), b.d["lens"], rot, shifts=shifts)
        ok()
        assert torch.equal(big[0][far:].view(torch.int16), near.view(torch.int16))
        del big, b


def test_windows_of_one_are_single_queries():
    lens = [37, 1, 200, 16]
    one = Batch(5, lens, None, 4, 2).cuda()
    win = Batch(5, lens, [1] * 4, 4, 2).cuda()
    a, la = one.call()
    w, lw = win.call()
    ok()
    one.check(a, la)
    win.check(w, lw)


def test_a_key_that_a_query_does_not_see_never_reaches_it():
    # infinities and NaNs in the K and V rows of a window's later tokens
    lens, qs = [70, 35], [20, 7]
    b = Batch(3, lens, qs, 2, 2)
    clean = b.kc.clone(), b.vc.clone()
    for s, at, what in ((0, 60, float("nan")), (0, 69, float("inf")), (1, 34, float("-inf"))):
        blk = int(b.tables[s, at // BLOCK])
        b.kc[blk, :, at % BLOCK, 3::7] = what
        b.vc[blk, :, at % BLOCK, 1::5] = what
    b.cuda()
    out, lse = b.call()
    ok()
    dirty = b.kc, b.vc
    b.kc, b.vc = clean
    ref, rl, tol, ltol = R.attend(b.q, b.kc, b.vc, b.tables, lens, b.cu, SCALE, b.lambdas, b.weight,
                                  1e-5, 0.8)
    got, gl = out.cpu().double(), lse.cpu().double()
    # queries before the first bad row: window 0 from position 50, window 1 from 28
    fine = torch.zeros(b.T, dtype=torch.bool)
    fine[0:10] = True
    fine[20:26] = True
    assert ((got - ref).abs() <= tol)[fine].all()
    assert ((gl - rl).abs() <= ltol)[fine].all()
    assert (~torch.isfinite(got[~fine])).any()
    b.kc, b.vc = dirty


def test_one_maps_infinities_stay_out_of_the_other():
    # minus infinity in a K row of the first map hides the key from it; the second sees it
    b = Batch(9, [40], None, 2, 1)
    b.q = b.q.abs()
    blk = int(b.tables[0, 1])
    b.kc[blk, 0, 4] = float("-inf")
    b.cuda()
    out, lse = b.call(norm=False)
    ok()
    a = []
    v = torch.cat([R.rows_of(b.vc, b.tables[0], 40, h) for h in (0, 1)], 1)
    for h in (0, 1):
        k = R.rows_of(b.kc, b.tables[0], 40, h)
        z = SCALE * (k @ b.q[0, h].double())
        assert abs(float(lse[0, h]) - float(torch.logsumexp(z, 0))) < 1e-4
        a.append(torch.softmax(z, 0) @ v)
    ref = 0.8 * (a[0] - float(b.lambdas[0]) * a[1])
    assert ((out[0, 0].cpu().double() - ref).abs() <= 4 * R.UBF * v.abs().amax(0)).all()


def test_a_nan_score_reaches_its_rows_alone():
    for lens in ([64, 48], [2500, 48]):
        b = Batch(13, lens, None, 2, 2)
        b.q[0, 0, 5] = float("nan")   # first map of head 0 of sequence 0
        b.cuda()
        out, lse = b.call()
        ok()
        assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
        assert torch.isfinite(out[0, 1]).all() and torch.isfinite(out[1]).all()
        assert torch.isfinite(lse[0, 1:]).all()


def test_a_difference_of_zero():
    # equal maps and lambda 1: with an eps the norm gives 0, without one too
    b = Batch(2, [33], None, 2, 1)
    b.kc[:, 1] = b.kc[:, 0]
    b.q[:, 1] = b.q[:, 0]
    b.lambdas.fill_(1.0)
    b.cuda()
    for eps in (1e-5, 0.0):
        out, _ = b.call(eps=eps)
        ok()
        assert (out[:b.T] == 0).all()
    # windows: of a segment that one worker has, both maps go the same way; of one that
    # ranges cut, each map at places of its own, so that weights are rounded to bf16
    # against other references (2^-8 of each at most, in either map): the difference is
    # then that of two roundings, which is what the bounds say of it
    for lens, qs in (([130], [70]), ([4000], [100])):
        b = Batch(2, lens, qs, 2, 1)
        b.kc[:, 1] = b.kc[:, 0]
        b.q[:, 1] = b.q[:, 0]
        b.lambdas.fill_(1.0)
        b.cuda()
        for norm in (False, True):
            out, _ = b.call(norm=norm, eps=0.0 if lens[0] == 130 else 1e-5)
            ok()
            if lens[0] == 130:
                assert (out[:b.T] == 0).all()
            else:
                b.check(out, None, norm=norm)


def test_many_sequences_and_a_wide_table():
    g = torch.Generator().manual_seed(1)
    lens = [int(x) for x in torch.randint(0, 60, (400,), generator=g)]
    b = Batch(17, lens, None, 2, 1, width=64).cuda()
    out, lse = b.call()
    ok()
    b.check(out, lse)


def test_bad_tables_contexts_and_windows_are_flagged():
    b = Batch(6, [40, 30], [4, 3], 2, 2).cuda()
    good, _ = b.call()
    ok()
    b.d["tables"][0, 1] = b.kc.shape[0]
    out, _ = b.call()
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_BLOCK_RANGE
    assert torch.equal(out[4:7].view(torch.int16), good[4:7].view(torch.int16))
    b.d["tables"][0, 1] = b.tables[0, 1]
    b.d["lens"][0] = 3                      # a window of 4 over 3 keys
    out, lse = b.call()
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_QLEN_RANGE
    assert (out[:4] == 3).all() and (lse[:4] == 5).all()
    assert torch.equal(out[4:7].view(torch.int16), good[4:7].view(torch.int16))
    b.d["lens"][0] = 49                     # past the table
    b.call()
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() & B.PA_DEVERR_CONTEXT_RANGE


def test_two_streams_and_a_graph():
    a = Batch(31, [700, 33, 90], None, 4, 2).cuda()
    c = Batch(32, [50, 600], [9, 17], 4, 2).cuda()
    wa, wc = a.call()[0], c.call()[0]
    ok()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (one, two):
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        with torch.cuda.stream(one):
            got.append((a.call()[0], wa))
        with torch.cuda.stream(two):
            got.append((c.call()[0], wc))
    ok()
    for x, want in got:
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))
    # captured and replayed on other inputs
    d = a.d
    out = torch.empty((a.T, a.hq // 2, 2 * DIM), dtype=torch.bfloat16, device="cuda")
    sh = B.shape_of(d["q"], d["kc"], d["tables"])
    ws = B.workspace(B.pa_decode_diff_workspace_size(sh, a.T), "cuda")
    call = B.prepare_decode_diff(d["q"], d["kc"], d["vc"], d["tables"], d["lens"], SCALE,
                                 d["lambdas"], out, norm_weight=d["weight"], out_scale=0.8,
                                 workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    other = Batch(33, [100, 690, 1], None, 4, 2)
    other.tables, other.kc, other.vc = a.tables.clone(), a.kc, a.vc
    other.lens = [400, 20, 70]
    d["q"].copy_(other.q)
    d["lens"].copy_(torch.tensor(other.lens, dtype=torch.int32))
    d["lambdas"].copy_(other.lambdas)
    d["weight"].copy_(other.weight)
    graph.replay()
    ok()
    other.check(out, None)


def test_a_layer_rotates_caches_and_attends():
    """Queries and keys rotated on their way into the cache, then read by
    differential attention: a prompt's window, then a step of single queries."""
    g = torch.Generator().manual_seed(41)
    hq, hkv, lens = 8, 4, [37, 90]
    per = [(n + 1 + BLOCK - 1) // BLOCK for n in lens]
    blocks = sum(per)
    ids = torch.randperm(blocks, generator=g).to(torch.int32)
    tables = torch.zeros((2, max(per)), dtype=torch.int32)
    tables[0, :per[0]], tables[1, :per[1]] = ids[:per[0]], ids[per[0]:]
    kc = torch.zeros((blocks, hkv, BLOCK, DIM), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rot = B.make_rotation(64, interleaved=True)
    b = Batch(1, lens, lens, hkv, hq // hkv)
    for new, ctx in ((lens, lens), ([1, 1], [n + 1 for n in lens])):
        T = sum(new)
        mixed = randn(g, T, hq + 2 * hkv, DIM).cuda()
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(new))
        pos = torch.cat([torch.arange(c - n, c) for n, c in zip(new, ctx)])
        slots = (tables[seq, pos // BLOCK].long() * BLOCK + pos % BLOCK).cuda()
        q = torch.empty((T, hq, DIM), dtype=torch.bfloat16, device="cuda")
        B.pa_rotate_and_cache(mixed[:, hq:hq + hkv], mixed[:, hq + hkv:], pos.int().cuda(), slots,
                              rot, kc, vc, q=mixed[:, :hq], q_out=q)
        ref, err = rotate_ref.rotate(mixed[:, :hq].cpu(), pos[:, None], rotate_ref.theta(64)[0], True)
        assert ((q.cpu().double() - ref).abs() <= rotate_ref.held_bf16(ref, err)).all()
        b.lens, b.qs, b.tables, b.kc, b.vc, b.q = ctx, new, tables, kc.cpu(), vc.cpu(), q.cpu()
        b.cu = torch.tensor([0, new[0], T], dtype=torch.int32)
        b.T, b.max_q = T, max(new)
        if max(new) == 1:
            b.qs = None
        b.cuda()
        out, lse = b.call()
        ok()
        b.check(out, lse)
