"""8-bit rows whose largest magnitude is tiny, in the oracle."""
import numpy as np
import pytest
import torch

from oracle import oracle


def tiny_rows():
    """Rows with zeros beside a largest magnitude of 2^-126 .. 2^-112: below 448 / FLT_MAX
    (2^-119.2) and 127 / FLT_MAX (2^-121.0) the factor to the codes is infinite in fp32."""
    x = torch.zeros(15, 128)
    for i in range(15):
        top = 2.0 ** (-126 + i)
        x[i, 3], x[i, 64], x[i, 127] = top, -top, max(top / 2, 2.0 ** -126)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["i8", "f8"])
def test_zeros_beside_a_tiny_value_stay_zeros(fmt):
    x = tiny_rows()
    codes, scales = getattr(oracle, f"quantize_rows_{fmt}")(x)
    codes, xf = np.asarray(codes), x.float().numpy()
    values = oracle.e4m3_values(codes) if fmt == "f8" else codes.astype(np.float64)
    assert np.isfinite(values).all() and np.isfinite(scales).all()
    assert (values[xf == 0] == 0).all()
    assert (np.abs(values * np.asarray(scales, np.float64)[:, None] - xf) <= 2.0 ** -119).all()
