"""8-bit rows whose largest magnitude is tiny, on their way into the cache."""
import numpy as np
import pytest
import torch

from oracle import oracle
from paged_kv_decode_18_gb300 import binding as B
from tests.rotate_ref import tiles_values
from tests.test_gpu_rotate import (BLOCK, DIM, KIND, _errors, _lib, empty_pool,  # noqa: F401
                                   ok, plain_write)
from tests.test_oracle_tiny_rows import tiny_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_zeros_beside_a_tiny_value_stay_zeros(fmt):
    x = tiny_rows()[:, None].cuda()
    slots = torch.arange(15, device="cuda")
    kc, vc = empty_pool(1, 1, fmt), empty_pool(1, 1, fmt)
    plain_write(x, x, slots, kc, vc, fmt)
    want, _ = getattr(oracle, {"int8": "quantize_rows_i8", "fp8": "quantize_rows_f8"}[fmt])(
        x[:, 0].cpu())
    got = kc[0, 0, :15 * DIM].cpu().numpy().reshape(15, DIM)
    assert np.array_equal(got, np.asarray(want).view(np.uint8))
    # the same on the way through a rotation: the values by any angle, the keys by none and by one
    for angle in (0.0, 0.7):
        kr, vr = empty_pool(1, 1, fmt), empty_pool(1, 1, fmt)
        B.pa_rotate_and_cache(x, x, torch.ones(15, dtype=torch.int32).cuda(), slots,
                              B.make_rotation_from([angle] * 64), kr, vr, kv_format=KIND[fmt])
        ok()
        assert torch.equal(vr, vc)
        if angle == 0.0:
            assert torch.equal(kr, kc)
        held = tiles_values(kr.cpu(), fmt)[0, 0, :15]
        # both sides of a pair are at most 2^-112 long; rows below 2^-117 may come back as zeros,
        # since their scales are subnormal
        assert torch.isfinite(held).all() and (held.abs() <= 2.0 ** -111).all()
        codes = kr[0, 0, :15 * DIM].cpu().view(15, DIM)
        zero = (x[:, 0].cpu() == 0) & (x[:, 0].cpu().roll(64, 1) == 0)
        assert ((codes & 0x7F)[zero] == 0).all()
    assert torch.equal(kc[0, 0, 15 * DIM:BLOCK * DIM], torch.full((DIM,), 0xA5, dtype=torch.uint8).cuda())
