"""pa_accumulate_weights on the GPU: windows of several query tiles called many
times over, whose tiles, issuing threads and epilogue groups meet in other ways
from call to call."""
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from tests.test_gpu_tree import same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    B.load()


@pytest.fixture(autouse=True)
def _errors():
    B.pa_debug_read_error()
    yield


def pool(fmt, blocks, hkv, g):
    if fmt == B.PA_KV_BF16:
        return torch.randn((blocks, hkv, 16, 128), generator=g).bfloat16().cuda()
    k = torch.randint(0, 256, (blocks, hkv, 2112), generator=g, dtype=torch.uint8)
    if fmt == B.PA_KV_FP8:
        k[..., :2048][(k[..., :2048] & 127) == 127] = 0     # no NaN codes
    scale = torch.rand((blocks, hkv, 16), generator=g) * 0.01
    k[..., 2048:] = scale.contiguous().view(torch.uint8)
    return k.cuda()


@pytest.mark.parametrize("fmt", [B.PA_KV_BF16, B.PA_KV_INT8, B.PA_KV_FP8])
@pytest.mark.parametrize("lens", [[1000, 1000], [130, 0, 64, 700, 1, 65, 300]])
def test_windows_of_several_tiles_many_times(fmt, lens):
    g = torch.Generator().manual_seed(51)
    ctx = [n + 900 + 37 * i for i, n in enumerate(lens)]
    blocks = [(c + 15) // 16 for c in ctx]
    tab = torch.zeros((len(ctx), max(blocks)), dtype=torch.int32)
    order, at = torch.randperm(sum(blocks), generator=g).int(), 0
    for s, n in enumerate(blocks):
        tab[s, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0] + lens).cumsum(0).int()
    q = torch.randn((int(cu[-1]), 8, 128), generator=g).bfloat16().cuda()
    lse = (torch.rand((int(cu[-1]), 8), generator=g) + 7).cuda()
    kc, tab, cu = pool(fmt, sum(blocks), 2, g), tab.cuda(), cu.cuda()
    c = torch.tensor(ctx, dtype=torch.int32).cuda()

    def call(weights):
        B.pa_accumulate_weights(q, kc, lse, tab, c, 0.088, weights, cu_seqlens_q=cu,
                                max_q_len=max(lens), accumulate=False, kv_format=fmt)

    first = torch.zeros((len(ctx), 2, max(ctx)), device="cuda")
    call(first)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == 0
    assert torch.isfinite(first).all() and (first > 0).any()
    many = [torch.zeros_like(first) for _ in range(50)]
    for w in many:
        call(w)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == 0
    for w in many:
        assert same_bits(w, first)


@pytest.mark.parametrize("fmt", [B.PA_KV_BF16, B.PA_KV_FP8])
@pytest.mark.parametrize("max_q", [8, 16, 700])   # mma.sync; tcgen05, one tile a window and several
@pytest.mark.parametrize("cu", [[0, 8, 11, 19], [0, 8, 8, 16], [0, 8, 5, 13], [0, 8, 40, 48]])
def test_windows_over_an_empty_context_are_flagged(fmt, max_q, cu):
    # the second sequence's context is empty: a window of queries, one of fewer than
    # none, or one outside the rows is not inside it; no query at all is
    g = torch.Generator().manual_seed(52)
    ctx = torch.tensor([60, 0, 33], dtype=torch.int32)
    tab = torch.arange(12, dtype=torch.int32).reshape(3, 4).cuda()
    q = torch.randn((19, 4, 128), generator=g).bfloat16().cuda()
    lse = torch.full((19, 4), 5.0, device="cuda")
    kc = pool(fmt, 12, 2, g)

    def call(offsets, lens):
        w = torch.full((3, 2, 64), 7.0, device="cuda")
        B.pa_accumulate_weights(q, kc, lse, tab, lens.cuda(), 0.088, w,
                                cu_seqlens_q=None if offsets is None else
                                torch.tensor(offsets, dtype=torch.int32).cuda(),
                                max_q_len=max_q, kv_format=fmt)
        torch.cuda.synchronize()
        return w, B.pa_debug_read_error()

    w, err = call(cu, ctx)
    assert err == (0 if cu[1] == cu[2] else B.PA_DEVERR_QLEN_RANGE)
    assert (w[1] == 7).all()                       # nothing is written for it
    assert not (w[0, :, 52:60] == 7).any() and (w[0, :, 60:] == 7).all()
    if cu == [0, 8, 11, 19]:                       # the others are as without it
        alone, err = call([0, 8, 8, 8], ctx)
        assert err == 0 and same_bits(alone[0].contiguous(), w[0].contiguous())


def test_one_query_over_an_empty_context_is_no_error():
    g = torch.Generator().manual_seed(53)
    q = torch.randn((2, 4, 128), generator=g).bfloat16().cuda()
    w = torch.full((2, 2, 32), 7.0, device="cuda")
    for max_q in (1, 700):
        B.pa_accumulate_weights(q, pool(B.PA_KV_BF16, 4, 2, g), torch.zeros((2, 4), device="cuda"),
                                torch.arange(4, dtype=torch.int32).reshape(2, 2).cuda(),
                                torch.tensor([0, 20], dtype=torch.int32).cuda(), 0.088, w,
                                max_q_len=max_q)
        torch.cuda.synchronize()
        assert B.pa_debug_read_error() == 0
    assert (w[0] == 7).all() and (w[1, :, 20:] == 7).all()
