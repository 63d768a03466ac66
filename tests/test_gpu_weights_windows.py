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
