"""Differential attention at the limits of what a call announces, on the GPU."""
import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from tests import diff_ref as R
from tests.test_gpu_diff import SCALE, Batch, _errors, _lib, ok  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def check_rows(b, out, lse, rows, norm=True, gain=0.8):
    """The rows of a boolean mask, against 64 bits."""
    ref, rl, tol, ltol = R.attend(b.q, b.kc, b.vc, b.tables, b.lens, b.cu, SCALE, b.lambdas,
                                  b.weight if norm else None, 1e-5, gain)
    got, gl = out[:b.T].cpu().double(), lse[:b.T].cpu().double()
    assert ((got - ref).abs() <= tol)[rows].all()
    assert ((gl - rl).abs() <= ltol)[rows].all()


@pytest.mark.parametrize("lens,qs,G,max_q,width", [
    ([600, 300], [4, 2], 2, 2, 0),                     # a CTA to a segment
    ([5000, 300], [4, 2], 2, 2, 400),                  # cut over all warps, merged by segment
    ([3000] + [90] * 120, [4] + [2] * 120, 2, 2, 0),   # merged by boundary, four warps to a CTA
    ([3000] + [90] * 120, [8] + [1] * 120, 1, 1, 0),
    ([3000] + [90] * 120, [2] + [1] * 120, 4, 1, 0),
    ([400, 200, 90], [300, 70, 3], 2, 70, 0),          # tcgen05 tiles and warp tiles
    ([400, 200], [90, 50], 2, 70, 0),                  # as many rows as two windows of 70
    ([400, 200], [9, 3], 16, 5, 0),
])
def test_a_window_longer_than_announced_is_flagged(lens, qs, G, max_q, width):
    b = Batch(71 + G, lens, qs, 2, G, width=width).cuda()
    out, lse = b.call(max_q=max_q, ws_fill=0)
    torch.cuda.synchronize()
    assert B.pa_debug_read_error() == B.PA_DEVERR_QLEN_RANGE
    # its rows are left as they were, the others get their results
    n = qs[0]
    assert (out[:n] == 3).all() and (lse[:n] == 5).all()
    rest = torch.ones(b.T, dtype=torch.bool)
    rest[:n] = False
    check_rows(b, out, lse, rest)
    # announced, it is served
    out, lse = b.call()
    ok()
    b.check(out, lse)


@pytest.mark.parametrize("G,qs", [
    (8, [169 + 2 * i for i in range(81)]),               # 20,169 tokens
    (4, [8000, 7000, 6500, 5000, 4000, 2200, 900, 3]),   # 33,603
])
def test_unequal_long_windows(G, qs):
    lens = [n + 40 for n in qs]
    b = Batch(81, lens, qs, 2, G).cuda()
    sh = B.shape_of(b.d["q"], b.d["kc"], b.d["tables"])
    assert B.pa_decode_diff_workspace_size(sh, b.T, b.max_q) > 0
    out, lse = b.call(ws_fill=0x7f)
    ok()
    if G == 8:
        b.check(out, lse)
        return
    # the same windows one by one (of the longest the 64-bit form would take minutes)
    for s in (0, 3, 6, 7):
        a, e = int(b.cu[s]), int(b.cu[s + 1])
        one = Batch.__new__(Batch)
        one.__dict__.update(b.__dict__)
        one.lens, one.qs, one.T, one.max_q = [lens[s]], [qs[s]], e - a, e - a
        one.cu = torch.tensor([0, e - a], dtype=torch.int32)
        one.d = dict(b.d, q=b.d["q"][a:e].contiguous(), cu=one.cu.cuda(),
                     tables=b.d["tables"][s:s + 1].contiguous(),
                     lens=torch.tensor([lens[s]], dtype=torch.int32).cuda())
        alone, la = one.call()
        ok()
        # weights rounded to bf16 against other references, then the output's own rounding
        far = (alone[:one.T].double() - out[a:e].double()).norm() / out[a:e].double().norm()
        assert float(far) < 1e-2
        assert (la - lse[a:e]).abs().max() < 1e-3


def test_tiles_that_32_bits_do_not_count_are_refused():
    # many heads under wide tables: only sizes are asked for
    def size(S, hq, hkv, width, T, max_q):
        sh = B.make_shape(num_seqs=S, num_q_heads=hq, num_kv_heads=hkv, head_dim=128,
                          block_size=16, max_blocks_per_seq=width, num_blocks=1024)
        return B.pa_decode_diff_workspace_size(sh, T, max_q)
    assert size(4096, 32, 32, (1 << 15) - 1, 4096, 1) > 0
    assert size(4096, 32, 32, 1 << 15, 4096, 1) == 0           # 4096 x 16 pairs x 2^15 tiles
    assert size(4000, 32, 32, 1 << 16, 4000, 1) == 0
    assert size(256, 64, 64, 1 << 20, 256, 1) == 0
    assert size(1, 16, 16, 1 << 26, 1, 1) == 0
    assert size(1000, 32, 32, 1 << 16, 64001, 64) == 0          # four query tiles to a window
    assert size(100, 32, 32, 1 << 16, 6401, 64) > 0


@pytest.mark.parametrize("S,q,G", [(900, None, 16), (850, 20, 2), (860, 1, 12)])
def test_a_long_plan_leaves_the_pair_kernel_two_stages(S, q, G):
    # beyond some 830 windows the third stage of K and V gives way to the plan
    lens = [(q or 0) + 7 * i % 300 for i in range(S)]
    b = Batch(96, lens, None if q is None else [q] * S, 2, G).cuda()
    out, lse = b.call(ws_fill=0xff)
    ok()
    b.check(out, lse)
    again, _ = b.call(with_lse=False, ws_fill=0)
    ok()
    assert torch.equal(again[:b.T].view(torch.int16), out[:b.T].view(torch.int16))


def most_sequences(words, pairs):
    """The most sequences whose plan fits: a word a pair and one at the end, three a
    sequence and two."""
    return (words - 3) // (pairs + 3)


def test_the_most_sequences_of_a_call():
    def size(S, G, T, max_q):
        sh = B.make_shape(num_seqs=S, num_q_heads=2 * G, num_kv_heads=2, head_dim=128,
                          block_size=16, max_blocks_per_seq=4, num_blocks=1024)
        return B.pa_decode_diff_workspace_size(sh, T, max_q)
    props = torch.cuda.get_device_properties(0)
    room = props.shared_memory_per_block_optin
    # warp tiles: a ring of 160 KB with 10 barriers, its alignment, 1 KB of weights
    words = (room - 160 * 1024 - 80 - 2048) // 4
    for G, max_q, pairs in ((1, 1, 1), (8, 1, 1), (8, 3, 3), (2, 15, 4), (4, 7, 4)):
        S = most_sequences(words, pairs)
        assert size(S, G, S * max_q - (max_q > 1), max_q) > 0, (G, max_q)
        S += 1
        assert size(S, G, S * max_q - (max_q > 1), max_q) == 0, (G, max_q)
    # pair kernel: two query tiles, two stages of 48 KB, 4864 bytes beside them, alignment; the
    # cut's words, one a pair of SMs
    words = (room - 1024 - 160 * 1024 - 4864) // 16 * 4 - props.multi_processor_count // 2 - 1
    S = (words - 4) // 4
    assert size(S, 16, S, 1) > 0 and size(S + 1, 16, S + 1, 1) == 0


def test_a_call_of_the_most_sequences():
    S = most_sequences((torch.cuda.get_device_properties(0).shared_memory_per_block_optin
                        - 160 * 1024 - 80 - 2048) // 4, 1)
    b = Batch(97, [5 * i % 37 for i in range(S)], None, 2, 1).cuda()
    out, lse = b.call(ws_fill=0x7f)
    ok()
    b.check(out, lse)
