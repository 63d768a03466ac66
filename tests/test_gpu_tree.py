"""Verifying a tree of drafted tokens on the GPU: the ancestor mask, attention
under it and the commit of the accepted path, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from paged_kv_decode_18_gb300 import workloads as W
from tests import tree_ref as R
from tests.gpu_util import DeviceBatch, Int8Batch

pytestmark = pytest.mark.gpu


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


# ---------------------------------------------------------------------------
# pa_tree_mask
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,words", [
    ([1], 1), ([7, 7, 7, 7], 1), ([3, 0, 32, 1, 33], 2), ([64, 5, 0, 61], 3), ([257], 9),
])
def test_mask_of_random_trees(lens, words):
    g = torch.Generator().manual_seed(1)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    parents = R.random_parents(g, lens)
    T = len(parents)
    ref, depths = R.tree_mask(parents, cu, words)
    mask = torch.full((T, words), 0x55555555, dtype=torch.int32, device="cuda")
    d = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    B.pa_tree_mask(parents.cuda(), torch.from_numpy(cu).cuda(), max(lens), mask, d)
    ok()
    assert np.array_equal(mask.cpu().numpy(), ref)
    assert np.array_equal(d.cpu().numpy(), depths)
    again = torch.zeros_like(mask)
    B.pa_tree_mask(parents.cuda(), torch.from_numpy(cu).cuda(), 32 * words, again)
    ok()
    assert torch.equal(mask, again)


@pytest.mark.parametrize("n", [400, 9000])
def test_mask_of_long_windows(n):
    # 400: a chain; 9000: more parents than shared memory holds, each node's
    # parent n/2 places before it
    parents = torch.arange(n, dtype=torch.int32) - 1 if n == 400 else \
        torch.where(torch.arange(n) < n // 2, torch.full((n,), -1), torch.arange(n) - n // 2).int()
    words = (n + 31) // 32
    mask = torch.zeros((n, words), dtype=torch.int32, device="cuda")
    d = torch.zeros((n,), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32)
    B.pa_tree_mask(parents.cuda(), cu.cuda(), n, mask, d)
    ok()
    ref, depths = R.tree_mask(parents, cu, words)
    assert np.array_equal(mask.cpu().numpy(), ref)
    assert np.array_equal(d.cpu().numpy(), depths)


def test_mask_bad_parents_and_windows_are_flagged():
    parents = torch.tensor([-1, 1, 0, -5, 2, 9, -1, 0], dtype=torch.int32)
    cu = torch.tensor([0, 6, 8], dtype=torch.int32)
    mask = torch.zeros((8, 1), dtype=torch.int32, device="cuda")
    B.pa_tree_mask(parents.cuda(), cu.cuda(), 6, mask)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_TREE_RANGE
    # nodes 1 (its own parent), 3 and 5 count as roots
    ref, _ = R.tree_mask(np.array([-1, -1, 0, -1, 2, -1, -1, 0]), cu.numpy(), 1)
    assert np.array_equal(mask.cpu().numpy(), ref)
    # a window longer than max_q_len keeps its rows as they were
    mask.fill_(77)
    B.pa_tree_mask(torch.full((8,), -1, dtype=torch.int32, device="cuda"), cu.cuda(), 5, mask)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_QLEN_RANGE
    assert (mask[:6] == 77).all() and mask[6:, 0].tolist() == [1, 2]


# ---------------------------------------------------------------------------
# pa_decode_tree
# ---------------------------------------------------------------------------

def tree_call(db, mask, max_q=None, with_lse=True, fill=0xA5):
    out = torch.full_like(db.q, 3.0)
    lse = torch.full(db.q.shape[:2], 3.0, dtype=torch.float32, device="cuda") if with_lse else None
    sh = B.shape_of(db.q, db.kc, db.block_tables)
    mq = max_q or db.w.max_q_len
    ws = B.workspace(B.pa_decode_tree_workspace_size(sh, db.q.shape[0], mq))
    ws.fill_(fill)
    B.pa_decode_tree(db.q, db.kc, db.vc, db.block_tables, db.context_lens, db.cu_seqlens_q,
                     mask, mq, db.w.scale, out, lse, workspace=ws)
    return out, lse


def reference(db, mask):
    w = db.w
    return R.tree_attention(w.q, db.kc.cpu(), db.vc.cpu(), w.block_tables, w.context_lens,
                            w.cu_seqlens_q, mask.cpu().numpy(), w.scale)


def random_mask(g, w, words, density):
    """Any bits, those past the windows included; some rows empty."""
    bits = torch.rand((w.num_q_tokens, words, 32), generator=g) < density
    bits[torch.rand((w.num_q_tokens,), generator=g) < 0.2] = False
    word = (bits.long() << torch.arange(32)).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).int()


# (query heads, KV heads, contexts, window lengths): one 16-row warp tile, and
# the 128-row tcgen05 tile with one and several tiles to a window
SHAPES = [
    (16, 8, [1, 17, 300, 16, 33], [1, 5, 8, 0, 7]),
    (8, 8, [16, 40, 129], [16, 9, 1]),
    (6, 2, [50, 5, 200], [5, 5, 3]),          # groups of 3: a padding row in the warp tile
    (10, 2, [64, 31], [3, 1]),                # 5
    (14, 2, [128, 2], [2, 2]),                # 7
    (32, 2, [100, 1, 260], [1, 1, 1]),        # 16: one token a tile
    (16, 8, [40, 300, 777, 130, 64], [40, 33, 9, 0, 64]),
    (6, 2, [140, 500, 43], [130, 50, 43]),    # 42 tokens a tile, two padding rows
    (16, 2, [70, 333], [20, 17]),             # 8
    (20, 1, [90, 17], [13, 1]),               # 20: six tokens a tile
    (128, 1, [129, 15], [3, 2]),              # a token fills the tile
]


@pytest.mark.parametrize("hq,hkv,ctx,ql", SHAPES)
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_tree_attention(hq, hkv, ctx, ql, kind):
    w = W.build("tree", 7, ctx, ql, pool_factor=1.3, num_q_heads=hq, num_kv_heads=hkv,
                outlier_frac=0.02)
    g = torch.Generator().manual_seed(8)
    words = (max(ql) + 31) // 32 + (kind == "any")
    if kind == "tree":
        mask = torch.from_numpy(R.tree_mask(R.random_parents(g, ql), w.cu_seqlens_q, words)[0])
    else:
        mask = random_mask(g, w, words, 0.4)
    db = DeviceBatch(w)
    out, lse = tree_call(db, mask.cuda())
    ok()
    R.assert_tree_close(out, lse, reference(db, mask), f"{hq}/{hkv} {kind}")
    # no lse, a larger bound (the same kernel's or the other's), another workspace content
    out2, _ = tree_call(db, mask.cuda(), max_q=32 * words, with_lse=False, fill=0)
    ok()
    R.assert_tree_close(out2, None, reference(db, mask), f"{hq}/{hkv} {kind} larger bound")


def test_long_context_in_many_pieces():
    for ql in ([5], [64]):
        w = W.build("cut", 9, [5000], ql, pool_factor=1.1, num_q_heads=4, num_kv_heads=2)
        g = torch.Generator().manual_seed(9)
        mask = torch.from_numpy(R.tree_mask(R.random_parents(g, ql), w.cu_seqlens_q, 2)[0])
        db = DeviceBatch(w)
        out, lse = tree_call(db, mask.cuda())
        ok()
        R.assert_tree_close(out, lse, reference(db, mask), f"pieces {ql}")
        again, lse2 = tree_call(db, mask.cuda(), fill=0)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_a_chain_equals_the_causal_window():
    w = W.build("chain", 10, [400, 90, 1000], [9, 64, 33], pool_factor=1.2)
    mask = torch.from_numpy(R.tree_mask(np.concatenate([np.arange(n) - 1 for n in (9, 64, 33)]),
                                        w.cu_seqlens_q, 2)[0]).cuda()
    db = DeviceBatch(w)
    out, lse = tree_call(db, mask)
    o2, l2 = db.varlen()
    ok()
    ref = reference(db, mask)
    R.assert_tree_close(out, lse, ref, "tree")
    R.assert_tree_close(o2, l2, ref, "causal")


@pytest.mark.parametrize("ctx,ql", [([40, 21], [8, 3]), ([700, 64, 150], [64, 64, 20]),
                                    ([16, 130], [8, 8]), ([3000, 1000], [8, 6]),
                                    ([3000, 1000], [64, 40])])
def test_infinities_and_nans_reach_only_those_who_see_them(ctx, ql):
    w = W.build("poison", 11, ctx, ql, pool_factor=1.2)
    g = torch.Generator().manual_seed(12)
    words = (max(ql) + 31) // 32
    mask = random_mask(g, w, words, 0.3)
    db = DeviceBatch(w)
    # K of one window row and V of others, in one KV head each
    for s in range(len(ctx)):
        def row(i):
            p = ctx[s] - ql[s] + i
            return int(w.block_tables[s, p // 16]), p % 16
        b, o = row(0)
        db.kc[b, 1, o, 5] = float("nan")
        b, o = row(ql[s] - 1)
        db.vc[b, 2, o, 7] = float("inf")
        db.vc[b, 2, o, 8] = float("-inf")
        db.vc[b, 2, o, 100] = float("nan")
        b, o = row(1)
        db.vc[b, 2, o, 7] = float("-inf")
        db.vc[b, 3, o] = 1e38
    ref = reference(db, mask)
    # a NaN score makes its whole row a NaN: out is compared there by the NaN alone
    out, lse = tree_call(db, mask.cuda())
    ok()
    sees_nan = torch.isnan(ref[0]).all(-1)
    assert sees_nan.any() and not sees_nan.all()
    got = out.cpu().double()
    assert torch.isnan(got[sees_nan]).all() and torch.isnan(lse.cpu()[sees_nan]).all()
    rest = ~sees_nan
    R.assert_tree_close(got[rest], lse.cpu()[rest], tuple(x[rest] for x in ref), "poison")


def test_bad_windows_blocks_and_contexts_are_flagged():
    w = W.build("bad", 13, [60, 100, 30], [8, 8, 8], pool_factor=1.2)
    db = DeviceBatch(w)
    mask = torch.full((24, 1), -1, dtype=torch.int32, device="cuda")
    ref = reference(db, mask)
    for what, flag in [("context", B.PA_DEVERR_QLEN_RANGE), ("long", B.PA_DEVERR_CONTEXT_RANGE),
                       ("block", B.PA_DEVERR_BLOCK_RANGE)]:
        for mq in (8, 32):    # both kernels
            lens, tab = db.context_lens.clone(), db.block_tables.clone()
            if what == "context":
                db.context_lens[1] = 5
            elif what == "long":
                db.context_lens[1] = 1 << 20
            else:
                db.block_tables[1, 0] = 1 << 20
            out, lse = tree_call(db, mask, max_q=mq)
            torch.cuda.synchronize()
            assert B.pa_debug_read_error() & flag, what
            db.context_lens.copy_(lens)
            db.block_tables.copy_(tab)
            rows = [i for i in range(24) if not 8 <= i < 16]
            R.assert_tree_close(out[rows], lse[rows], tuple(x[rows] for x in ref), what)
            if what == "context":   # produces no rows
                assert (out[8:16] == 3.0).all() and (lse[8:16] == 3.0).all()


def test_tree_call_in_a_graph_and_on_another_stream():
    ql = [12, 3, 40]
    w = W.build("graph", 14, [300, 50, 200], ql, pool_factor=1.2)
    db = DeviceBatch(w)
    g = torch.Generator().manual_seed(15)
    parents = R.random_parents(g, ql).cuda()
    mask = torch.zeros((sum(ql), 2), dtype=torch.int32, device="cuda")
    out = torch.empty_like(db.q)
    lse = torch.empty(db.q.shape[:2], dtype=torch.float32, device="cuda")
    sh = B.shape_of(db.q, db.kc, db.block_tables)
    ws = B.workspace(B.pa_decode_tree_workspace_size(sh, sum(ql), 40))

    def step():
        B.pa_tree_mask(parents, db.cu_seqlens_q, 40, mask)
        B.pa_decode_tree(db.q, db.kc, db.vc, db.block_tables, db.context_lens, db.cu_seqlens_q,
                         mask, 40, w.scale, out, lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    ok()
    R.assert_tree_close(out, lse, reference(db, mask), "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (16, 17):
        parents.copy_(R.random_parents(torch.Generator().manual_seed(seed), ql))
        db.q.copy_(torch.randn(db.q.shape, generator=g).bfloat16())
        db.w.q = db.q.cpu()
        out.fill_(9.0)
        graph.replay()
        ok()
        R.assert_tree_close(out, lse, reference(db, mask), f"replay {seed}")


# ---------------------------------------------------------------------------
# pa_commit_path
# ---------------------------------------------------------------------------

def moved_by_hand(pool, tables, ctx, ql, paths):
    """The pool after every row of every path has moved, through a copy."""
    got = pool.clone()
    rows = pool if pool.dim() == 4 else None

    def place(s, p):
        return int(tables[s, p // 16]), p % 16
    for s, path in enumerate(paths):
        for i, j in enumerate(path):
            (b0, o0), (b1, o1) = (place(s, ctx[s] - ql[s] + x) for x in (j, i))
            if rows is not None:
                got[b1, :, o1] = pool[b0, :, o0]
            else:
                got[b1, :, o1 * 128:(o1 + 1) * 128] = pool[b0, :, o0 * 128:(o0 + 1) * 128]
                got[b1, :, 2048 + o1 * 4:2052 + o1 * 4] = pool[b0, :, 2048 + o0 * 4:2052 + o0 * 4]
    return got


def same_bits(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hkv", [1, 8, 11])
def test_commit(fmt, hkv):
    ctx, ql = [8, 40, 100, 300, 33, 64], [8, 7, 64, 50, 0, 64]
    paths = [[2, 5, 7], [0, 1, 2], list(range(1, 64, 2)), [], [], list(range(64))]
    paths[3] = sorted(torch.randperm(50, generator=torch.Generator().manual_seed(1))[:21].tolist())
    w = W.build("commit", 18, ctx, ql, pool_factor=1.2, num_q_heads=hkv, num_kv_heads=hkv)
    db = DeviceBatch(w) if fmt == "bf16" else Int8Batch(w, fp8=fmt == "fp8")
    tab, lens = w.block_tables.cuda(), w.context_lens.cuda()
    path = torch.full((6, 64), 1 << 30, dtype=torch.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    kref = moved_by_hand(db.kc.cpu(), w.block_tables, ctx, ql, paths)
    vref = moved_by_hand(db.vc.cpu(), w.block_tables, ctx, ql, paths)
    cu = w.cu_seqlens_q.cuda()
    # the new lengths in the place of the old
    B.pa_commit_path(db.kc, db.vc, tab, lens, cu, path.cuda(), n.cuda(), lens)
    ok()
    assert same_bits(db.kc, kref) and same_bits(db.vc, vref)
    assert lens.tolist() == [c - q + len(p) for c, q, p in zip(ctx, ql, paths)]


@pytest.mark.parametrize("path,n", [([3, 2], 2), ([1, 1], 2), ([-1, 2], 2), ([0, 8], 2),
                                    ([0, 1], 3), ([0, 1], -1)])
def test_commit_bad_paths_are_flagged_and_move_nothing(path, n):
    w = W.build("badpath", 19, [40, 20], [8, 4], pool_factor=1.2)
    db = DeviceBatch(w)
    k0, v0 = db.kc.clone(), db.vc.clone()
    rows = torch.tensor([path, [1, 3]], dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.pa_commit_path(db.kc, db.vc, db.block_tables, db.context_lens, db.cu_seqlens_q, rows,
                     torch.tensor([n, 2], dtype=torch.int32, device="cuda"), new)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_TREE_RANGE
    assert new.tolist() == [40, 18]
    other = moved_by_hand(k0.cpu(), w.block_tables, [40, 20], [8, 4], [[], [1, 3]])
    assert same_bits(db.kc, other)


def test_rows_past_four_gigabytes():
    # a pool of 4.6 GB; the sequence's blocks lie at its end
    NB, S = 140000, 2
    kc = torch.empty((NB, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-64:] = torch.randn((64, 8, 16, 128), device="cuda").bfloat16()
    vc[-64:] = torch.randn((64, 8, 16, 128), device="cuda").bfloat16()
    ids = NB - 1 - torch.randperm(60, generator=torch.Generator().manual_seed(1))
    tab = ids.reshape(2, 30).int()
    small = (tab - (NB - 64)).int()   # the same rows in a pool of the last 64 blocks
    lens, cu = [470, 333], torch.tensor([0, 40, 47], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((47, 16, 128), generator=g).bfloat16()
    mask = torch.from_numpy(R.tree_mask(R.random_parents(g, [40, 7]), cu, 2)[0])
    for mq in (40, 8):
        if mq == 8:   # the warp tile: the second window alone
            q, mask, cu = q[40:], mask[40:], torch.tensor([0, 0, 7], dtype=torch.int32)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(q.shape[:2], device="cuda")
        sh = B.shape_of(out, kc, tab)
        ws = B.workspace(B.pa_decode_tree_workspace_size(sh, q.shape[0], mq))
        B.pa_decode_tree(q.cuda(), kc, vc, tab.cuda(), torch.tensor(lens).int().cuda(), cu.cuda(),
                         mask.cuda(), mq, 0.09, out, lse, workspace=ws)
        ok()
        ref = R.tree_attention(q, kc[-64:].cpu(), vc[-64:].cpu(), small, lens, cu, mask.numpy(),
                               0.09)
        R.assert_tree_close(out, lse, ref, "far blocks")
    ql, paths = [40, 7], [[1, 5, 17, 39], [2, 3, 6]]
    kref = moved_by_hand(kc[-64:].cpu(), small, lens, ql, paths)
    path = torch.tensor([[1, 5, 17, 39], [2, 3, 6, -1]], dtype=torch.int32, device="cuda")
    new = torch.zeros(S, dtype=torch.int32, device="cuda")
    B.pa_commit_path(kc, vc, tab.cuda(), torch.tensor(lens).int().cuda(),
                     torch.tensor([0, 40, 47]).int().cuda(), path,
                     torch.tensor([4, 3]).int().cuda(), new)
    ok()
    assert same_bits(kc[-64:], kref) and new.tolist() == [434, 329]
    assert math.prod(kc.shape) * 2 > 1 << 32


# ---------------------------------------------------------------------------
# sizes at which every ring of stages wraps and segments are cut, against 64-bit
# matrix products on the GPU
# ---------------------------------------------------------------------------

def dense_reference(w, kc, vc, mask):
    """tree_attention's results and tolerances as matrix products in 64 bits."""
    Tq, Hq, D = w.q.shape
    Hkv = w.num_kv_heads
    G = Hq // Hkv
    out = torch.zeros(Tq, Hq, D, dtype=torch.float64)
    tol, lse, ltol = torch.zeros_like(out), torch.zeros(Tq, Hq).double(), torch.zeros(Tq, Hq).double()
    q = w.q.cuda().double()
    for s in range(w.num_seqs):
        a, b, c = int(w.cu_seqlens_q[s]), int(w.cu_seqlens_q[s + 1]), int(w.context_lens[s])
        L = b - a
        if L == 0:
            continue
        hidden = torch.zeros(L, c, dtype=torch.bool)
        for j in range(L):
            hidden[j, c - L:] = ~R.bits_to_bool(mask[a + j].numpy(), L)
        hidden = hidden.cuda()
        ids = w.block_tables[s, :(c + 15) // 16].long().cuda()
        for h in range(Hkv):
            k = kc[ids, h].reshape(-1, D)[:c].double()
            v = vc[ids, h].reshape(-1, D)[:c].double()
            x = q[a:b, h * G:(h + 1) * G].transpose(0, 1)
            z = (w.scale * x @ k.T).masked_fill(hidden, float("-inf"))
            big = (w.scale * x.abs() @ k.abs().T).masked_fill(hidden, 0).amax(-1, keepdim=True)
            p = torch.softmax(z, -1)
            o, spread = p @ v, p @ v.abs()
            ez = 136 * R.U32 * big + 2.0 ** -21
            out[a:b, h * G:(h + 1) * G] = o.transpose(0, 1).cpu()
            tol[a:b, h * G:(h + 1) * G] = (R.UBF * (1 + R.UBF) * (o.abs() + spread)
                                           + 4 * ez * spread + 2.0 ** -30).transpose(0, 1).cpu()
            l = torch.logsumexp(z, -1)
            lse[a:b, h * G:(h + 1) * G] = l.T.cpu()
            ltol[a:b, h * G:(h + 1) * G] = (2 * ez[..., 0] + 4 * R.U32 * l.abs()).T.cpu()
    return out, lse, tol, ltol


@pytest.mark.parametrize("hq,hkv,ctx,ql", [
    (16, 8, [6001, 3333, 128, 5000, 40, 4097], [64, 40, 33, 64, 7, 64]),      # a tile a window
    (32, 4, [9000, 5555, 2500], [64, 61, 50]),                                # four: pairs of CTAs
    (24, 4, [4000, 8191, 700], [64, 64, 22]),                                 # groups of 6, two padding rows
    (16, 8, [8000, 3001, 17, 6400, 5], [8, 5, 8, 1, 3]),                      # warp tiles
    (16, 8, [300 + 37 * i for i in range(40)], [1 + i % 8 for i in range(40)]),
])
def test_large_batches(hq, hkv, ctx, ql):
    w = W.build("large", 20, ctx, ql, pool_factor=1.1, num_q_heads=hq, num_kv_heads=hkv,
                outlier_frac=0.01)
    g = torch.Generator().manual_seed(21)
    mask = torch.from_numpy(R.tree_mask(R.random_parents(g, ql), w.cu_seqlens_q, 2)[0])
    db = DeviceBatch(w)
    ref = dense_reference(w, db.kc, db.vc, mask)
    out, lse = tree_call(db, mask.cuda())
    ok()
    R.assert_tree_close(out, lse, ref, f"large {hq}/{hkv}")
    out2, lse2 = tree_call(db, mask.cuda(), fill=0)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_two_streams_at_once():
    # two batches, each call with its own workspace, interleaved on two streams
    ql = [[64, 40], [8, 3]]
    ws, dbs, masks = [], [], []
    for i in range(2):
        w = W.build("two", 22 + i, [3000, 1500], ql[i], pool_factor=1.1)
        g = torch.Generator().manual_seed(24)
        dbs.append(DeviceBatch(w))
        masks.append(torch.from_numpy(R.tree_mask(R.random_parents(g, ql[i]), w.cu_seqlens_q, 2)[0]))
        ws.append(w)
    refs = [dense_reference(w, db.kc, db.vc, m) for w, db, m in zip(ws, dbs, masks)]
    dm = [m.cuda() for m in masks]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = tree_call(dbs[i], dm[i])
    ok()
    for i in range(2):
        R.assert_tree_close(*got[i], refs[i], f"stream {i}")
