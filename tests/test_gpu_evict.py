"""Accumulated attention weight and eviction on the GPU against plain forms:
the weights to 64 bits, what stays and where it lies bit for bit; and the
operators in a row, as a serving loop runs them."""
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from paged_kv_decode_18_gb300 import workloads as W
from tests import tree_ref as R
from tests.gpu_util import DeviceBatch, Int8Batch
from tests.test_gpu_tree import same_bits

pytestmark = pytest.mark.gpu

FORMATS = {"bf16": B.PA_KV_BF16, "int8": B.PA_KV_INT8, "fp8": B.PA_KV_FP8}


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


def rows_of(pool, fmt, tables, lens):
    """(s, h) -> the cached K rows in 64 bits, dequantised."""
    pool = pool.cpu()

    def rows(s, h):
        c = int(lens[s])
        ids = tables[s, :(c + 15) // 16].long()
        t = pool[ids, h]
        if fmt == "bf16":
            return t.reshape(-1, 128)[:c].double()
        code = t[:, :2048].contiguous()
        code = code.view(torch.int8).double() if fmt == "int8" else \
            code.view(torch.float8_e4m3fn).float().double()
        scale = t[:, 2048:].contiguous().view(torch.float32).double()
        return (code.reshape(-1, 16, 128) * scale.reshape(-1, 16, 1)).reshape(-1, 128)[:c]
    return rows


def batch(w, fmt):
    return DeviceBatch(w) if fmt == "bf16" else Int8Batch(w, fp8=fmt == "fp8")


def some_lse(w, rows):
    """A log-sum-exp for every query: the causal window's own."""
    Hkv, G = w.num_kv_heads, w.num_q_heads // w.num_kv_heads
    lse = torch.full((w.num_q_tokens, w.num_q_heads), float("-inf"))
    for s in range(w.num_seqs):
        a, b, c = int(w.cu_seqlens_q[s]), int(w.cu_seqlens_q[s + 1]), int(w.context_lens[s])
        for h in range(Hkv if b > a else 0):
            z = w.scale * torch.einsum("jgd,pd->jgp", w.q[a:b, h * G:(h + 1) * G].double(),
                                       rows(s, h))
            see = torch.arange(c) <= (c - (b - a) + torch.arange(b - a))[:, None]
            lse[a:b, h * G:(h + 1) * G] = torch.logsumexp(
                z.masked_fill(~see[:, None], float("-inf")), -1).float()
    return lse


def weights_call(db, w, fmt, lse, weights, add, cu=True, max_q=None):
    B.pa_accumulate_weights(w.q.cuda(), db.kc, lse.cuda(), w.block_tables.cuda(),
                            w.context_lens.cuda(), w.scale, weights,
                            cu_seqlens_q=w.cu_seqlens_q.cuda() if cu else None,
                            max_q_len=max_q or max(1, w.max_q_len), accumulate=add,
                            kv_format=FORMATS[fmt])


WINDOWS = [
    (16, 8, [1, 16, 17, 300, 33], [1, 1, 1, 1, 1]),
    (8, 8, [40, 5, 129], [9, 5, 0]),
    (6, 2, [70, 500], [33, 1]),
    (32, 2, [260, 2], [3, 2]),            # 16 heads a KV head: two groups of columns a query
    (4, 2, [700, 64, 200], [150, 64, 65]),
    (24, 1, [150], [40]),
    (16, 8, [1000, 130], [64, 64]),
]


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hq,hkv,ctx,ql", WINDOWS)
def test_weights(fmt, hq, hkv, ctx, ql):
    w = W.build("weights", 31, ctx, ql, pool_factor=1.2, num_q_heads=hq, num_kv_heads=hkv,
                outlier_frac=0.03, outlier_gain=3.0)
    db = batch(w, fmt)
    rows = rows_of(db.kc, fmt, w.block_tables, w.context_lens)
    lse = some_lse(w, rows)
    lse[0, 0] = float("-inf")    # a query that saw nothing
    n = max(ctx) + 5
    old = torch.rand((len(ctx), hkv, n), generator=torch.Generator().manual_seed(1))
    for s, (c, q) in enumerate(zip(ctx, ql)):
        old[s, :, c - q:] = float("nan")   # the window's own and what lies past the context
    for add in (True, False):
        got = old.cuda()
        weights_call(db, w, fmt, lse, got, add)
        ok()
        ref, tol = R.accumulate(w.q, rows, lse, ctx, w.cu_seqlens_q, w.scale, old, add, hkv)
        got = got.cpu()
        for s, c in enumerate(ctx):
            d = (got[s, :, :c].double() - ref[s, :, :c]).abs()
            assert (d - tol[s, :, :c]).max() <= 0, (add, s, float(d.max()))
            assert torch.isnan(got[s, :, c:]).all()
        twice = old.cuda()
        weights_call(db, w, fmt, lse, twice, add, max_q=4096)
        ok()
        assert torch.allclose(twice.cpu(), got, rtol=1e-5, atol=1e-9, equal_nan=True)
        again = old.cuda()
        weights_call(db, w, fmt, lse, again, add)
        assert same_bits(again, got.contiguous())
    if set(ql) == {1}:
        one = old.cuda()
        weights_call(db, w, fmt, lse, one, False, cu=False)
        ok()
        assert same_bits(one, got)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hq,hkv,ql", [(16, 8, 1), (8, 8, 2), (16, 8, 7), (16, 8, 64), (4, 4, 300)])
def test_weights_of_large_batches(fmt, hq, hkv, ql):
    # sizes at which every ring of stages wraps, against 64-bit matrix products on
    # the GPU; two sequences have windows of their own lengths
    ctx = [4100, 2500, 311, 6007, 900, 1]
    lens = [min(ql, c) for c in ctx]
    lens[1], lens[4] = max(1, lens[1] // 2), 0
    check_large(fmt, hq, hkv, ctx, lens)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (6, 2), (8, 1)])
def test_weights_of_windows_of_one_and_several_query_tiles(fmt, hq, hkv):
    check_large(fmt, hq, hkv, [4100, 3000, 311, 6007, 900, 1, 513, 2048],
                [1, 300, 64, 200, 0, 1, 513, 65])


def check_large(fmt, hq, hkv, ctx, lens):
    w = W.build("large", 44, ctx, lens, pool_factor=1.1, num_q_heads=hq, num_kv_heads=hkv,
                outlier_frac=0.02, outlier_gain=2.5)
    db = batch(w, fmt)
    rows = rows_of(db.kc, fmt, w.block_tables, w.context_lens)
    G = hq // hkv
    old = torch.rand((len(ctx), hkv, 6007), generator=torch.Generator().manual_seed(3)) * 0.01
    lse = torch.zeros((w.num_q_tokens, hq))
    ref, tol = old.double(), torch.zeros(old.shape, dtype=torch.float64)
    for s, c in enumerate(ctx):
        a, L = int(w.cu_seqlens_q[s]), lens[s]
        hidden = (torch.arange(c) > (c - L + torch.arange(L))[:, None]).cuda()
        for h in range(hkv if L else 0):
            k = rows(s, h).cuda()
            x = w.q[a:a + L, h * G:(h + 1) * G].cuda().double().transpose(0, 1)
            z = (w.scale * x @ k.T).masked_fill(hidden, float("-inf"))
            l = torch.logsumexp(z, -1).float()
            lse[a:a + L, h * G:(h + 1) * G] = l.T.cpu()
            l = l.double()[..., None]
            p = torch.exp(z - l)
            err = p * (140 * R.U32 * (w.scale * x.abs() @ k.abs().T) + 8 * R.U32 *
                       (z.masked_fill(hidden, 0).abs() + l.abs()) + 2.0 ** -20)
            tot, e = p.sum((0, 1)).cpu(), err.sum((0, 1)).cpu()
            before = old[s, h, :c].double()
            before[c - L:] = 0
            ref[s, h, :c] = before + tot
            tol[s, h, :c] = 2 * e + L * G * R.U32 * tot + 2 * R.U32 * (before + tot) + 1e-37
    got = old.cuda()
    weights_call(db, w, fmt, lse, got, True)
    ok()
    d = (got.cpu().double() - ref).abs()
    assert (d <= tol).all(), float((d - tol).max())
    again = old.cuda()
    weights_call(db, w, fmt, lse, again, True)
    assert same_bits(again, got)


@pytest.mark.parametrize("mq", [1, 512])
def test_weights_bad_windows_are_flagged_and_keep_theirs(mq):
    ctx, ql = [60, 100, 30], [8, 8, 8]
    w = W.build("bad", 32, ctx, ql, pool_factor=1.2)
    db = batch(w, "bf16")
    rows = rows_of(db.kc, "bf16", w.block_tables, ctx)
    lse = some_lse(w, rows)
    old = torch.rand((3, 8, 112), generator=torch.Generator().manual_seed(2))
    ref, tol = R.accumulate(w.q, rows, lse, ctx, w.cu_seqlens_q, w.scale, old, True, 8)
    lens = w.context_lens.clone()
    w.context_lens[1] = 7
    got = old.cuda()
    weights_call(db, w, "bf16", lse, got, True, max_q=8 * mq)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_QLEN_RANGE
    assert torch.equal(got[1].cpu(), old[1])
    for s in (0, 2):
        assert ((got[s].cpu().double() - ref[s]).abs() <= tol[s] + 0).all()
    # a context longer than the weights' rows
    w.context_lens.copy_(lens)
    short = torch.zeros((3, 8, 64), device="cuda")
    weights_call(db, w, "bf16", lse, short, True, max_q=8 * mq)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() & B.PA_DEVERR_CONTEXT_RANGE
    # block ids outside the pool
    w.block_tables[2, 1] = -1
    got = old.cuda()
    weights_call(db, w, "bf16", lse, got, True, max_q=8 * mq)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() & B.PA_DEVERR_BLOCK_RANGE
    assert ((got[0].cpu().double() - ref[0]).abs() <= tol[0]).all()


# ---------------------------------------------------------------------------
# pa_evict
# ---------------------------------------------------------------------------

def evict_by_hand(pools, weights, tables, ctx, budgets, most, sinks, recent):
    """Pools and weights after every head's rows have moved through a copy, and
    the positions; entries past the new lengths are None'd by the caller."""
    got = [p.clone() for p in pools]
    w = weights.clone()
    S, H, _ = weights.shape
    kept = torch.full((S, H, most), -1, dtype=torch.int32)
    for s in range(S):
        for h in range(H):
            stay = R.evict_positions(weights[s, h], ctx[s], budgets[s], sinks, recent)
            kept[s, h, :len(stay)] = torch.tensor(stay, dtype=torch.int32)
            src = torch.tensor(stay, dtype=torch.long)
            dst = torch.arange(len(stay))
            w[s, h, :len(stay)] = weights[s, h, src]
            b0, o0 = tables[s].long()[src // 16], src % 16
            b1, o1 = tables[s].long()[dst // 16], dst % 16
            for p, q in zip(pools, got):
                if p.dim() == 4:
                    q[b1, h, o1] = p[b0, h, o0]
                else:
                    f, t = p[..., :2048].unflatten(-1, (16, 128)), q[..., :2048].unflatten(-1, (16, 128))
                    t[b1, h, o1] = f[b0, h, o0]
                    f, t = p[..., 2048:].unflatten(-1, (16, 4)), q[..., 2048:].unflatten(-1, (16, 4))
                    t[b1, h, o1] = f[b0, h, o0]
    return got, w, kept


def check_evict(fmt, ctx, budgets, most, sinks, recent, weights, hkv=8, seed=33):
    w = W.build("evict", seed, ctx, [min(1, c) for c in ctx], pool_factor=1.2, num_q_heads=hkv,
                num_kv_heads=hkv)
    db = batch(w, fmt)
    lens, tab = w.context_lens.cuda(), w.block_tables.cuda()
    pools = (db.kc.cpu(), db.vc.cpu())
    (kref, vref), wref, kept = evict_by_hand(pools, weights, w.block_tables, ctx, budgets, most,
                                             sinks, recent)
    got_w = weights.cuda()
    got_kept = torch.full((len(ctx), hkv, most), 99, dtype=torch.int32, device="cuda")
    new = torch.full((len(ctx),), 99, dtype=torch.int32, device="cuda")
    B.pa_evict(db.kc, db.vc, tab, lens, got_w, torch.tensor(budgets, dtype=torch.int32).cuda(),
               sinks, recent, got_kept, new)
    ok()
    n = [min(c, b) for c, b in zip(ctx, budgets)]
    assert new.tolist() == n
    assert torch.equal(got_kept.cpu(), kept)
    for s in range(len(ctx)):
        # the weights of what stays, and everything past the old context
        assert same_bits(got_w[s, :, :n[s]].contiguous(), wref[s, :, :n[s]].contiguous())
        assert same_bits(got_w[s, :, ctx[s]:].contiguous(), weights[s, :, ctx[s]:].contiguous())
    # every row of the new caches, and every row of the blocks that hold none
    used = torch.zeros(w.pool_shape()[0], 16, dtype=torch.bool)
    for s in range(len(ctx)):
        p = torch.arange(n[s], ctx[s])
        used[w.block_tables[s].long()[p // 16], p % 16] = True   # unspecified afterwards
    for got, ref in ((db.kc.cpu(), kref), (db.vc.cpu(), vref)):
        if got.dim() == 4:
            a, b = got.view(torch.int16).permute(0, 2, 1, 3), ref.view(torch.int16).permute(0, 2, 1, 3)
            assert torch.equal(a[~used], b[~used])
        else:
            for lo, hi, n_ in ((0, 2048, 128), (2048, 2112, 4)):
                a = got[..., lo:hi].unflatten(-1, (16, n_)).permute(0, 2, 1, 3)
                b = ref[..., lo:hi].unflatten(-1, (16, n_)).permute(0, 2, 1, 3)
                assert torch.equal(a[~used], b[~used])


def heavy(g, S, H, n):
    u = torch.rand((S, H, n), generator=g)
    return torch.where(u < 0.2, torch.zeros(()), 0.02 / (1.001 - u))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 16), (1, 0), (0, 31)])
def test_evict(fmt, sinks, recent):
    ctx = [100, 33, 600, 47, 1, 1300, 64]
    budgets = [50, 40, 100, 47, 47, 1000, 63]
    g = torch.Generator().manual_seed(34)
    check_evict(fmt, ctx, budgets, 1000, sinks, recent, heavy(g, 7, 8, 1310))


@pytest.mark.parametrize("kind", ["equal", "few", "odd", "sorted", "negative"])
def test_evict_ties_and_odd_weights(kind):
    g = torch.Generator().manual_seed(35)
    x = torch.rand((3, 2, 700), generator=g)
    if kind == "equal":
        x.fill_(0.25)
    elif kind == "few":
        x = (x * 4).floor() / 4
    elif kind == "odd":
        for v in (float("nan"), float("inf"), float("-inf"), -0.0, 0.0, 1e-42, -1e-42):
            x[torch.rand(x.shape, generator=g) < 0.15] = v
    elif kind == "sorted":
        x = x.sort(-1).values
    else:
        x = -x
    # 1e-42 is below fp32's normal range; a key is its bits, so it counts as it is
    check_evict("bf16", [700, 300, 513], [333, 17, 512], 512, 2, 5, x, hkv=2)


def test_evict_to_nothing_and_protected_only():
    g = torch.Generator().manual_seed(36)
    check_evict("bf16", [100, 20], [0, 0], 3, 0, 0, heavy(g, 2, 2, 100), hkv=2)
    check_evict("bf16", [100, 20, 12], [12, 12, 12], 12, 5, 7, heavy(g, 3, 2, 112), hkv=2)


def test_evict_long_context():
    g = torch.Generator().manual_seed(37)
    check_evict("bf16", [20011, 9000], [4096, 8999], 8999, 4, 512, heavy(g, 2, 1, 20016), hkv=1)
    check_evict("fp8", [12345], [12000], 12000, 0, 0, heavy(g, 1, 2, 12352), hkv=2)


def test_evict_many_heads():
    # more (sequence, KV head) pairs than fill the GPU: one CTA each, many waves
    g = torch.Generator().manual_seed(45)
    ctx = [900 - 11 * i for i in range(20)]
    for fmt in ("bf16", "int8"):
        check_evict(fmt, ctx, [c - 200 + 7 * (i % 5) for i, c in enumerate(ctx)], 800, 2, 100,
                    heavy(g, 20, 8, 912))


def test_evict_slices_longer_than_shared_memory():
    g = torch.Generator().manual_seed(46)
    x = heavy(g, 1, 1, 170011)
    x[0, 0, ::3] = 0.25
    check_evict("bf16", [170011], [60001], 60001, 4, 1000, x, hkv=1)


def test_evict_bad_values_are_flagged_and_change_nothing():
    ctx = [100, 100, 100]
    w = W.build("badev", 38, ctx, [1] * 3, pool_factor=1.2)
    for what, flag in [("budget", B.PA_DEVERR_BUDGET_RANGE), ("large", B.PA_DEVERR_BUDGET_RANGE),
                       ("context", B.PA_DEVERR_CONTEXT_RANGE), ("minus", B.PA_DEVERR_CONTEXT_RANGE),
                       ("block", B.PA_DEVERR_BLOCK_RANGE)]:
        db = batch(w, "bf16")
        k0 = db.kc.clone()
        g = torch.Generator().manual_seed(39)
        x = heavy(g, 3, 8, 112)
        got = x.cuda()
        budgets = torch.tensor([50, 50, 50], dtype=torch.int32)
        lens, tab = w.context_lens.clone(), w.block_tables.clone()
        if what == "budget":
            budgets[1] = 19
        elif what == "large":
            budgets[1] = 61
        elif what == "context":
            lens[1] = 113
        elif what == "minus":
            lens[1] = -1
        else:
            tab[1, :] = 1 << 25
        kept = torch.zeros((3, 8, 60), dtype=torch.int32, device="cuda")
        new = torch.zeros(3, dtype=torch.int32, device="cuda")
        B.pa_evict(db.kc, db.vc, tab.cuda(), lens.cuda(), got, budgets.cuda(), 4, 16, kept, new)
        torch.cuda.synchronize()
        assert B.pa_debug_read_error() == flag, what
        assert new.tolist()[0] == 50 and new.tolist()[2] == 50
        mine = w.block_tables[1, :7].long().cuda()
        assert same_bits(db.kc[mine], k0[mine])
        if what != "block":
            assert new[1] == lens[1] and (kept[1] == -1).all()
            assert torch.equal(got[1].cpu(), x[1])


def test_evict_and_weights_past_four_gigabytes():
    NB = 140000
    kc = torch.empty((NB, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-64:] = torch.randn((64, 8, 16, 128), device="cuda").bfloat16()
    vc[-64:] = torch.randn((64, 8, 16, 128), device="cuda").bfloat16()
    tab = (NB - 1 - torch.randperm(60, generator=torch.Generator().manual_seed(1))).reshape(2, 30).int()
    small = (tab - (NB - 64)).int()
    ctx = [470, 333]
    g = torch.Generator().manual_seed(40)
    w0 = torch.zeros((2, 8, 480))
    for ql in ([1, 1], [70, 64]):
        q = torch.randn((sum(ql), 16, 128), generator=g).bfloat16()
        lse = torch.full((sum(ql), 16), 6.0)
        cu = torch.tensor([0, ql[0], sum(ql)], dtype=torch.int32)
        got = w0.cuda()
        B.pa_accumulate_weights(q.cuda(), kc, lse.cuda(), tab.cuda(), torch.tensor(ctx).int().cuda(),
                                0.08, got, cu_seqlens_q=cu.cuda(), max_q_len=max(ql))
        ok()
        ref, tol = R.accumulate(q, rows_of(kc[-64:], "bf16", small, ctx), lse, ctx, cu, 0.08, w0,
                                True, 8)
        assert ((got.cpu().double() - ref).abs() <= tol).all()
    x = heavy(g, 2, 8, 480)
    (kref, vref), _, kept = evict_by_hand((kc[-64:].cpu(), vc[-64:].cpu()), x, small, ctx,
                                          [200, 100], 200, 4, 16)
    got_kept = torch.zeros((2, 8, 200), dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.pa_evict(kc, vc, tab.cuda(), torch.tensor(ctx).int().cuda(), x.cuda(),
               torch.tensor([200, 100]).int().cuda(), 4, 16, got_kept, new)
    ok()
    assert torch.equal(got_kept.cpu(), kept) and new.tolist() == [200, 100]
    for s in range(2):
        ids = small[s, :6].long()
        assert same_bits(kc[-64:][ids.cuda()], kref[ids]) and same_bits(vc[-64:][ids.cuda()], vref[ids])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_a_serving_step_verify_commit_weigh_evict_decode():
    """Drafted trees are verified and their accepted paths committed; the accepted
    queries' weights are added, the caches shrink, and a decode over what is
    left equals attention over the rows that should be left. Once in order,
    once captured and replayed on another stream."""
    ctx, ql = [300, 150, 64], [20, 7, 33]
    w = W.build("step", 41, ctx, ql, pool_factor=1.3)
    g = torch.Generator().manual_seed(42)
    parents = R.random_parents(g, ql)
    ref_mask, depths = R.tree_mask(parents, w.cu_seqlens_q, 2)
    # accept the path to each tree's deepest node
    paths, rows = [], []
    for s in range(3):
        a, b = int(w.cu_seqlens_q[s]), int(w.cu_seqlens_q[s + 1])
        j, path = a + int(depths[a:b].argmax()) - a, []
        while j >= 0:
            path.insert(0, j)
            j = int(parents[a + j])
        paths.append(path)
        rows += [a + p for p in path]
    path = torch.full((3, 16), -1, dtype=torch.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    cu2 = torch.cat([torch.zeros(1), n.cumsum(0)]).int()
    db = DeviceBatch(w)
    k0, v0 = db.kc.clone(), db.vc.clone()
    tq = sum(ql)
    mask = torch.zeros((tq, 2), dtype=torch.int32, device="cuda")
    weights = torch.zeros((3, 8, 320), device="cuda")
    weights.copy_(torch.rand((3, 8, 320), generator=g) * 0.01)
    w0 = weights.clone()
    out, lse = torch.empty_like(db.q), torch.empty((tq, 16), device="cuda")
    sh = B.shape_of(db.q, db.kc, db.block_tables)
    ws = B.workspace(B.pa_decode_tree_workspace_size(sh, tq, 33))
    ws2 = B.workspace(B.pa_decode_workspace_size(sh, 0))
    lens, lens2 = db.context_lens.clone(), torch.zeros_like(db.context_lens)
    budgets = torch.tensor([128, 100, 48], dtype=torch.int32, device="cuda")
    kept = torch.zeros((3, 8, 128), dtype=torch.int32, device="cuda")
    q2 = torch.randn((3, 16, 128), generator=g).bfloat16().cuda()
    out2, lse2 = torch.empty_like(q2), torch.empty((3, 16), device="cuda")
    par, path, n, cu2 = parents.cuda(), path.cuda(), n.cuda(), cu2.cuda()
    pick = torch.tensor(rows, device="cuda")

    def step():
        B.pa_tree_mask(par, db.cu_seqlens_q, 33, mask)
        B.pa_decode_tree(db.q, db.kc, db.vc, db.block_tables, lens, db.cu_seqlens_q, mask, 33,
                         w.scale, out, lse, workspace=ws)
        B.pa_commit_path(db.kc, db.vc, db.block_tables, lens, db.cu_seqlens_q, path, n, lens)
        B.pa_accumulate_weights(db.q[pick], db.kc, lse[pick], db.block_tables, lens, w.scale,
                                weights, cu_seqlens_q=cu2, max_q_len=16)
        B.pa_evict(db.kc, db.vc, db.block_tables, lens, weights, budgets, 4, 24, kept, lens2)
        B.pa_decode(q2, db.kc, db.vc, db.block_tables, lens2, w.scale, out2, lse2, workspace=ws2)

    def check(what):
        ok()
        kp, vp = k0.cpu(), v0.cpu()
        R.assert_tree_close(out, lse, R.tree_attention(
            w.q, kp, vp, w.block_tables, ctx, w.cu_seqlens_q, ref_mask, w.scale), what)
        for s in range(3):
            p0 = ctx[s] - ql[s]
            left = list(range(p0)) + [p0 + j for j in paths[s]]   # old positions, in order
            assert int(lens[s]) == len(left)
            m = min(len(left), int(budgets[s]))
            assert int(lens2[s]) == m
            for h in range(8):
                k = R.cached(kp, w.block_tables[s], ctx[s], h)[left]
                v = R.cached(vp, w.block_tables[s], ctx[s], h)[left]
                got = kept[s, h, :m].cpu().long()
                assert (got[1:] > got[:-1]).all() and got[:4].tolist() == list(range(4))
                # the weights say the same choice, up to what lies within rounding of the border
                one = w0[s, h].cpu().clone()
                c, L = len(left), len(paths[s])
                for j, node in enumerate(paths[s]):
                    for gq in range(2):
                        row = int(w.cu_seqlens_q[s]) + node
                        z = w.scale * (k[:c - L + j + 1] @ w.q[row, 2 * h + gq].double())
                        p = torch.exp(z - torch.logsumexp(z, 0)).float()
                        if j == 0 and gq == 0:
                            one[c - L:c] = 0
                        one[:c - L + j + 1] += p
                want = R.evict_positions(one, c, m, 4, 24)
                differ = set(want) ^ set(got.tolist())
                border = one[want[4:m - 24]].min() if m < c else 0
                assert all(abs(one[x] - border) < 1e-5 for x in differ), what
                for gq in range(2):
                    z = w.scale * (k[got] @ q2[s, 2 * h + gq].cpu().double())
                    pr = torch.softmax(z, 0)
                    o = pr @ v[got]
                    err = (out2[s, 2 * h + gq].cpu().double() - o).abs()
                    assert (err <= R.UBF * o.abs() + 1e-4 * (pr @ v[got].abs()) + 1e-6).all(), what
    step()
    check("in order")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step()
    for t in range(2):
        db.kc.copy_(k0), db.vc.copy_(v0), weights.copy_(w0), lens.copy_(db.context_lens)
        out.zero_(), out2.zero_(), kept.zero_(), mask.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        check(f"replay {t}")


