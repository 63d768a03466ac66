"""Block tables as wide as a serving engine's context limit: the entries past a
sequence's context are never looked at, whatever they hold. The tree call
chooses another kernel for such a table, the others the same or another cluster."""
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from paged_kv_decode_18_gb300 import workloads as W
from tests import tree_ref as R
from tests.gpu_util import DeviceBatch
from tests.test_gpu_evict import FORMATS, batch, heavy
from tests.test_gpu_tree import reference, same_bits, tree_call

pytestmark = pytest.mark.gpu

WIDTH = 4096     # 65536 positions


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


def widened(tab, ctx):
    """The table with entries outside the pool behind every context."""
    t = torch.full((tab.shape[0], WIDTH), -1, dtype=torch.int32)
    t[:, 1::2] = 1 << 25
    for s, c in enumerate(ctx):
        n = (c + 15) // 16
        t[s, :n] = tab[s, :n]
    return t.cuda()


@pytest.mark.parametrize("hq,hkv,ctx,ql", [
    (16, 8, [128, 200, 301, 384], [7, 7, 7, 7]),       # one row tile
    (16, 8, [128, 200, 301, 384], [12, 9, 12, 12]),    # two: the tcgen05 tile by the table's width
    (6, 2, [140, 500, 43], [130, 50, 43]),
])
def test_tree_attention(hq, hkv, ctx, ql):
    w = W.build("wide", 61, ctx, ql, pool_factor=1.3, num_q_heads=hq, num_kv_heads=hkv)
    g = torch.Generator().manual_seed(62)
    mask = torch.from_numpy(R.tree_mask(R.random_parents(g, ql), w.cu_seqlens_q,
                                        (max(ql) + 31) // 32)[0])
    db = DeviceBatch(w)
    ref = reference(db, mask)
    db.block_tables = widened(w.block_tables, ctx)
    out, lse = tree_call(db, mask.cuda())
    ok()
    R.assert_tree_close(out, lse, ref, "wide table")


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("ql", [1, 20, 150])
def test_weights(fmt, ql):
    ctx = [700, 150, 333]
    w = W.build("wide", 63, ctx, [ql] * 3, pool_factor=1.2, num_q_heads=8, num_kv_heads=4)
    db = batch(w, fmt)
    g = torch.Generator().manual_seed(64)
    lse = (torch.rand((3 * ql, 8), generator=g) + 6).cuda()
    old = torch.rand((3, 4, 700), generator=g)
    got = []
    for tab in (w.block_tables.cuda(), widened(w.block_tables, ctx)):
        x = old.cuda()
        B.pa_accumulate_weights(w.q.cuda(), db.kc, lse, tab, w.context_lens.cuda(), w.scale, x,
                                cu_seqlens_q=w.cu_seqlens_q.cuda(), max_q_len=ql,
                                kv_format=FORMATS[fmt])
        ok()
        got.append(x)
    assert same_bits(got[0], got[1])
    assert not same_bits(got[0], old)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_commit_and_evict(fmt):
    ctx, ql = [300, 47, 900], [20, 7, 33]
    w = W.build("wide", 65, ctx, ql, pool_factor=1.2)
    g = torch.Generator().manual_seed(66)
    x = heavy(g, 3, 8, 900)
    path = torch.tensor([[0, 3, 9], [1, 2, 5], [4, 20, 32]], dtype=torch.int32).cuda()
    n = torch.tensor([3, 2, 3], dtype=torch.int32).cuda()
    got = []
    for wide in (False, True):
        db = batch(w, fmt)
        tab = widened(w.block_tables, ctx) if wide else w.block_tables.cuda()
        lens = w.context_lens.cuda()
        B.pa_commit_path(db.kc, db.vc, tab, lens, w.cu_seqlens_q.cuda(), path, n, lens)
        weights, new = x.cuda(), torch.zeros_like(lens)
        kept = torch.zeros((3, 8, 400), dtype=torch.int32, device="cuda")
        budgets = torch.tensor([64, 50, 400], dtype=torch.int32, device="cuda")
        B.pa_evict(db.kc, db.vc, tab, lens, weights, budgets, 2, 30, kept, new)
        ok()
        assert lens.tolist() == [283, 42, 870] and new.tolist() == [64, 42, 400]
        rows = []
        for s, m in enumerate(new.tolist()):
            ids = w.block_tables[s, :(m + 15) // 16].long().cuda()
            for pool in (db.kc, db.vc):
                t = pool[ids]
                parts = [t] if fmt == "bf16" else [t[..., :2048].unflatten(-1, (16, 128)),
                                                   t[..., 2048:].unflatten(-1, (16, 4))]
                rows += [p.transpose(1, 2).flatten(0, 1)[:m].contiguous() for p in parts]
            rows.append(weights[s, :, :m].contiguous())
        got.append(rows + [kept])
    for a, b in zip(*got):
        assert same_bits(a, b)
