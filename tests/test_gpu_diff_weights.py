"""The softmax weights of differential attention's single queries, where the two
maps nearly agree: what is left of them is then all that their weights' errors
can hide."""
import math

import pytest
import torch

from tests.diff_ref import DIM, U32, UBF, rows_of
from tests.test_gpu_diff import SCALE, Batch, _errors, _lib, ok  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

# A weight enters the product as its upper eight bits and what they leave, less than 2^-7 of
# it, rounded by half a step: 2^-15 of it.
WEIGHT = 2.0 ** -7 * UBF


def attend(b, gain):
    """A row's output without a norm in 64 bits, and its bound: as in diff_ref, but for
    the weights."""
    out = torch.zeros(b.T, b.hq // 2, 2 * DIM, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for s, c in enumerate(b.lens):
        for p in range(b.hkv // 2):
            v = torch.cat([rows_of(b.vc, b.tables[s], c, 2 * p + i) for i in (0, 1)], 1)
            for g in range(b.G):
                lam = float(b.lambdas[p * b.G + g])
                d, ed = 0.0, 0.0
                for i, factor in ((0, 1.0), (1, -lam)):
                    x = b.q[s, (2 * p + i) * b.G + g].double()
                    k = rows_of(b.kc, b.tables[s], c, 2 * p + i)
                    dz = (128 + 4) * U32 * SCALE * float((k.abs() @ x.abs()).max()) + 2.0 ** -21
                    w = torch.softmax(SCALE * (k @ x), 0)
                    a, mass = w @ v, w @ v.abs()
                    d = d + factor * a
                    ed = ed + abs(factor) * ((math.expm1(2 * dz) + WEIGHT + (c + 64) * U32) * mass
                                             + 4 * U32 * a.abs())
                out[s, p * b.G + g] = gain * d
                ed = abs(gain) * ed
                tol[s, p * b.G + g] = ed + UBF * (abs(gain) * d.abs() + ed) + 2.0 ** -126
    return out, tol


@pytest.mark.parametrize("lens,hkv,G,width", [
    ([2, 9, 17, 33], 4, 1, 0), ([7, 12, 5], 2, 4, 0), ([9, 16, 30], 2, 3, 0),   # a CTA to a segment
    ([6, 11, 21], 2, 5, 0), ([8, 15], 4, 8, 0),
    ([2, 9, 17, 33], 4, 1, 400), ([7, 12, 40], 2, 4, 400), ([8, 15], 4, 8, 400),  # cut, by segment
    ([3 + i % 20 for i in range(200)], 2, 2, 0), ([3 + i % 9 for i in range(160)], 2, 6, 0),
    ([900, 2500], 2, 2, 0), ([1800], 2, 7, 0),                                   # merged
])
def test_nearly_equal_maps(lens, hkv, G, width):
    b = Batch(91 + G, lens, None, hkv, G, width=width)
    # the second map's queries and keys are the first's, the queries a little longer
    b.kc[:, 1::2] = b.kc[:, 0::2]
    q = b.q.view(b.T, hkv // 2, 2, G, DIM)
    q[:, :, 1] = (q[:, :, 0].float() * 1.02).to(torch.bfloat16)
    b.lambdas.fill_(1.0)
    b.cuda()
    out, _ = b.call(norm=False, gain=8.0)
    ok()
    ref, tol = attend(b, 8.0)
    err = (out[:b.T].cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


def test_an_infinite_value_is_none_but_itself():
    # 0 x infinity is a NaN: neither part of a weight may be 0 beside one. Lambda below 0, so
    # that both maps' infinities have one sign
    for width in (0, 400):
        for lens, G in (([20], 2), ([3], 6), ([700], 4)):
            b = Batch(95, lens, None, 2, G, width=width)
            # one key far above the others: its weight is 1, a bf16 number
            b.kc[int(b.tables[0, 0]), :, 1] *= 4
            b.vc[int(b.tables[0, 0]), 0, 1, 7] = float("inf")
            b.vc[int(b.tables[0, 0]), 1, 0, 9] = float("-inf")
            b.lambdas.fill_(-0.5)
            b.cuda()
            out, _ = b.call(norm=False)
            ok()
            got = out[0].cpu().float()
            assert (got[:, 7] == math.inf).all() and (got[:, DIM + 9] == -math.inf).all()
            rest = torch.ones(2 * DIM, dtype=torch.bool)
            rest[7] = rest[DIM + 9] = False
            assert torch.isfinite(got[:, rest]).all()
