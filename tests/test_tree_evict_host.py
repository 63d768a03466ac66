"""Tree verification and eviction without a GPU: the C entry points refuse bad
arguments before anything touches a device, the binding refuses tensors that
do not fit, and the plain forms agree with each other."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from tests import tree_ref as R

P = ctypes.c_void_p(0x10000)   # never dereferenced: every case fails host checks
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def shape(**kw):
    base = dict(num_seqs=4, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16,
                max_blocks_per_seq=24, num_blocks=128)
    base.update(kw)
    return B.make_shape(**base)


def test_tree_mask_refusals(lib):
    def call(parents=P, cu=P, S=4, T=28, mq=7, mask=P, words=1, depths=P):
        return lib.pa_tree_mask(parents, cu, S, T, mq, mask, words, depths, None)
    assert call(S=-1) == B.PA_ERR_ARG
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(T=1 << 31) == B.PA_ERR_ARG
    assert call(mq=-1) == B.PA_ERR_ARG
    assert call(mq=33) == B.PA_ERR_ARG          # does not fit one word
    assert call(words=-1) == B.PA_ERR_ARG
    assert call(words=(1 << 20) + 1) == B.PA_ERR_ARG
    assert call(mq=0) == B.PA_ERR_ARG           # rows, but no window may hold them
    assert call(parents=None) == B.PA_ERR_ARG
    assert call(cu=None) == B.PA_ERR_ARG
    assert call(mask=None) == B.PA_ERR_ARG
    assert call(parents=ODD) == B.PA_ERR_ARG
    assert call(depths=ODD) == B.PA_ERR_ARG
    assert call(S=0) == B.PA_OK
    assert call(T=0, parents=None, mask=None) == B.PA_OK


def test_decode_tree_refusals(lib):
    def call(sh=None, q=P, mask=P, words=1, T=28, mq=7, out=P, ws=P, n=1 << 40, scale=0.1):
        sh = sh or shape()
        return lib.pa_decode_tree(q, P, P, P, P, P, mask, words, T, mq, scale, out, None,
                                  ctypes.byref(sh), ws, n, None)
    assert call(shape(head_dim=64)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(block_size=32)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(num_q_heads=129, num_kv_heads=1)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(num_q_heads=12)) == B.PA_ERR_ARG
    assert call(shape(num_blocks=1 << 26)) == B.PA_ERR_UNSUPPORTED
    assert call(mq=33) == B.PA_ERR_ARG
    assert call(words=-1, mq=0) == B.PA_ERR_ARG
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(mq=-1) == B.PA_ERR_ARG
    assert call(mq=0) == B.PA_ERR_ARG
    assert call(q=None) == B.PA_ERR_ARG
    assert call(mask=None) == B.PA_ERR_ARG
    assert call(out=ODD) == B.PA_ERR_ARG
    assert call(mask=ODD) == B.PA_ERR_ARG
    assert call(scale=float("nan")) == B.PA_ERR_ARG
    assert call(shape(num_seqs=0)) == B.PA_OK
    assert call(T=0) == B.PA_OK
    assert lib.pa_decode_tree_workspace_size(ctypes.byref(shape(head_dim=64)), 28, 7) == 0
    assert lib.pa_decode_tree_workspace_size(ctypes.byref(shape()), 0, 7) == 0


def test_commit_path_refusals(lib):
    def call(sh=None, k=P, fmt=B.PA_KV_BF16, lens=P, path=P, most=4, new=ctypes.c_void_p(0x20000)):
        sh = sh or shape()
        return lib.pa_commit_path(k, P, fmt, P, lens, P, path, P, most, new, ctypes.byref(sh),
                                  None)
    assert call(shape(head_dim=64)) == B.PA_ERR_UNSUPPORTED
    assert call(fmt=3) == B.PA_ERR_ARG
    assert call(fmt=-1) == B.PA_ERR_ARG
    assert call(most=-1) == B.PA_ERR_ARG
    assert call(k=None) == B.PA_ERR_ARG
    assert call(k=ctypes.c_void_p(0x10008)) == B.PA_ERR_ARG
    assert call(path=None) == B.PA_ERR_ARG
    assert call(new=None) == B.PA_ERR_ARG
    assert call(new=ODD) == B.PA_ERR_ARG
    assert call(new=ctypes.c_void_p(0x10008)) == B.PA_ERR_ARG   # overlaps context_lens
    assert call(shape(num_seqs=0)) == B.PA_OK


def test_accumulate_weights_refusals(lib):
    def call(sh=None, q=P, k=P, fmt=B.PA_KV_BF16, lse=P, cu=P, T=28, mq=7, w=P, n=384, scale=.1):
        sh = sh or shape()
        return lib.pa_accumulate_weights(q, k, fmt, lse, P, P, cu, T, mq, scale, 1, w, n,
                                         ctypes.byref(sh), None)
    assert call(shape(head_dim=64)) == B.PA_ERR_UNSUPPORTED
    assert call(fmt=7) == B.PA_ERR_ARG
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(mq=-1) == B.PA_ERR_ARG
    assert call(n=-1) == B.PA_ERR_ARG
    assert call(cu=None) == B.PA_ERR_ARG        # 28 rows for 4 sequences
    assert call(q=None) == B.PA_ERR_ARG
    assert call(lse=None) == B.PA_ERR_ARG
    assert call(w=None) == B.PA_ERR_ARG
    assert call(q=ctypes.c_void_p(0x10004)) == B.PA_ERR_ARG
    assert call(w=ODD) == B.PA_ERR_ARG
    assert call(scale=float("nan")) == B.PA_ERR_ARG
    assert call(shape(num_seqs=0)) == B.PA_OK


def test_evict_refusals(lib):
    far = ctypes.c_void_p(0x20000)

    def call(sh=None, k=P, fmt=B.PA_KV_BF16, lens=P, w=P, n=384, most=64, sinks=4, recent=16,
             kept=P, new=far):
        sh = sh or shape()
        return lib.pa_evict(k, P, fmt, P, lens, w, n, P, most, sinks, recent, kept, new,
                            ctypes.byref(sh), None)
    assert call(shape(block_size=8)) == B.PA_ERR_UNSUPPORTED
    assert call(fmt=3) == B.PA_ERR_ARG
    assert call(n=-1) == B.PA_ERR_ARG
    assert call(most=-1) == B.PA_ERR_ARG
    assert call(sinks=-1) == B.PA_ERR_ARG
    assert call(recent=-1) == B.PA_ERR_ARG
    assert call(sinks=60, recent=5) == B.PA_ERR_ARG
    assert call(k=None) == B.PA_ERR_ARG
    assert call(kept=None) == B.PA_ERR_ARG
    assert call(new=P) == B.PA_ERR_ARG          # the lengths are read meanwhile
    assert call(new=ctypes.c_void_p(0x10004)) == B.PA_ERR_ARG
    assert call(kept=ODD) == B.PA_ERR_ARG
    assert call(shape(num_seqs=70000)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(num_seqs=0)) == B.PA_OK


def test_binding_refuses_host_tensors():
    i32 = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.pa_tree_mask(i32, i32, 4, torch.zeros(5, 1, dtype=torch.int32))
    pool = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    q = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    tab = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.pa_decode_tree(q, pool, pool, tab, i32[:4], i32, torch.zeros(5, 1, dtype=torch.int32),
                         4, 0.1, q)
    with pytest.raises(ValueError):
        B.pa_commit_path(pool, pool, tab, i32[:4], i32, tab, i32[:4], i32[:4])
    with pytest.raises(ValueError):
        B.pa_accumulate_weights(q, pool, torch.zeros(5, 2), tab, i32[:4], 0.1,
                                torch.zeros(4, 1, 32), cu_seqlens_q=i32, max_q_len=2)
    with pytest.raises(ValueError):
        B.pa_evict(pool, pool, tab, i32[:4], torch.zeros(4, 1, 32), i32[:4], 1, 1,
                   torch.zeros(4, 1, 8, dtype=torch.int32), i32[:4])


def test_reference_mask_is_the_closure_of_the_parents():
    g = torch.Generator().manual_seed(3)
    lens = [1, 5, 0, 40, 33]
    cu = np.concatenate([[0], np.cumsum(lens)])
    parents = R.random_parents(g, lens)
    mask, depths = R.tree_mask(parents, cu, 2)
    for s, n in enumerate(lens):
        up = np.zeros((n, n), int)
        for j in range(n):
            p = int(parents[cu[s] + j])
            if p >= 0:
                up[j, p] = 1
        closure, power = np.eye(n, dtype=int), np.eye(n, dtype=int)
        for _ in range(n):
            power = power @ up
            closure += power
        for j in range(n):
            assert np.array_equal(R.bits_to_bool(mask[cu[s] + j], n).numpy(), closure[j] > 0)
            assert depths[cu[s] + j] == closure[j].sum() - 1


def test_reference_of_a_chain_is_causal_attention():
    # one sequence, a chain of drafted tokens: torch's softmax over the causal keys
    g = torch.Generator().manual_seed(4)
    k = torch.randn(2, 1, 16, 128, generator=g).bfloat16()
    v = torch.randn(2, 1, 16, 128, generator=g).bfloat16()
    q = torch.randn(5, 2, 128, generator=g).bfloat16()
    tab = torch.tensor([[1, 0]], dtype=torch.int32)
    mask, _ = R.tree_mask(np.arange(5) - 1, [0, 5], 1)
    out, lse, _, _ = R.tree_attention(q, k, v, tab, [23], [0, 5], mask, 0.1)
    kk = torch.cat([k[1, 0], k[0, 0]])[:23].double()
    vv = torch.cat([v[1, 0], v[0, 0]])[:23].double()
    for j in range(5):
        z = 0.1 * q[j].double() @ kk[:19 + j].T
        assert torch.allclose(out[j], torch.softmax(z, -1) @ vv[:19 + j])
        assert torch.allclose(lse[j], torch.logsumexp(z, -1))


def test_reference_eviction_order():
    w = torch.tensor([9.0, 0.0, -0.0, 5.0, float("nan"), 5.0, float("-inf"), float("inf"), 1.0])
    assert R.evict_positions(w, 9, 9, 0, 0) == list(range(9))
    assert R.evict_positions(w, 9, 3, 0, 0) == [0, 3, 7]            # 5.0 twice: the first
    assert R.evict_positions(w, 9, 3, 1, 1) == [0, 7, 8]
    assert R.evict_positions(w, 9, 6, 0, 0) == [0, 1, 3, 5, 7, 8]   # 0 and -0 are equal
    assert R.evict_positions(w, 9, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8]  # the NaN goes first
    assert R.evict_positions(w, 9, 0, 0, 0) == []
