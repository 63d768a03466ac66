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
