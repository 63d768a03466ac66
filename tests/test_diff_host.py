"""Differential attention without a GPU: refusals of the C entry point and of
the binding."""
import ctypes

import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild

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


def test_refusals(lib):
    def call(sh=None, q=P, kc=P, vc=P, tables=P, lens=P, cu=P, T=28, mq=7, scale=0.1, lam=P, w=None,
             eps=1e-5, gain=1.0, out=P, lse=None, ws=P, n=1 << 40):
        return lib.pa_decode_diff(q, kc, vc, tables, lens, cu, T, mq, 1, scale, lam, w, eps, gain,
                                  out, lse, ctypes.byref(sh or shape()), ws, n, None)
    nan = float("nan")
    assert call(shape(head_dim=64)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(block_size=32)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(num_q_heads=7, num_kv_heads=7)) == B.PA_ERR_UNSUPPORTED  # no pairs
    assert call(shape(num_q_heads=258, num_kv_heads=2)) == B.PA_ERR_UNSUPPORTED
    assert call(shape(num_q_heads=12)) == B.PA_ERR_ARG
    assert call(shape(num_blocks=1 << 26)) == B.PA_ERR_UNSUPPORTED
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(T=1 << 31) == B.PA_ERR_ARG
    assert call(mq=-1) == B.PA_ERR_ARG
    assert call(mq=0) == B.PA_ERR_ARG
    assert call(cu=None) == B.PA_ERR_ARG              # 28 rows are not one per sequence
    assert call(cu=None, T=4, mq=2) == B.PA_ERR_ARG
    assert call(scale=nan) == B.PA_ERR_ARG
    assert call(eps=-1.0) == B.PA_ERR_ARG
    assert call(eps=nan) == B.PA_ERR_ARG
    assert call(gain=nan) == B.PA_ERR_ARG
    for name in ("q", "kc", "vc", "tables", "lens", "lam", "out"):
        assert call(**{name: None}) == B.PA_ERR_ARG, name
        assert call(**{name: ODD}) == B.PA_ERR_ARG, name
    assert call(w=ctypes.c_void_p(0x10004)) == B.PA_ERR_ARG
    assert call(lse=ODD) == B.PA_ERR_ARG
    assert call(shape(num_seqs=0)) == B.PA_OK
    assert call(T=0) == B.PA_OK
    size = lib.pa_decode_diff_workspace_size
    assert size(ctypes.byref(shape(num_q_heads=7, num_kv_heads=7)), 28, 7) == 0
    assert size(ctypes.byref(shape()), 0, 7) == 0
    assert size(ctypes.byref(shape()), 28, 0) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros((4, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.prepare_decode_diff(x, x, x, x, x, 0.1, x, x)
