"""Plain 64-bit forms of the rotary-position operators, written from their
definitions, and how far the kernels' roundings can take a result. They share
nothing with the library."""
import math

import torch

BLOCK, DIM = 16, 128
UBF = 2.0 ** -8    # half a step of bf16 (finfo.eps / 2)
# Cosine and sine: the phase is rounded to 2^-23 turns (2 pi 2^-24 = 3.7e-7 radians),
# and turned into radians below pi by an fp32 constant and one product (2 pi 2^-24 =
# 3.7e-7 together); the fast functions add 2^-21.1 = 4.5e-7. Together 1.2e-6 = 2^-19.7.
UCS = 2.0 ** -19.7


def theta(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """(angles per position, magnitude), a pair at a time."""
    got, magnitude = [], 1.0
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    for i in range(rot_dim // 2):
        t = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            t = t / factor
        elif scaling == "bands":
            n = original_len * t / (2 * math.pi)
            if n <= low:
                t = t / factor
            elif n < high:
                s = (n - low) / (high - low)
                t = t * s + t / factor * (1 - s)
        elif scaling == "ramp":
            def pair(turns):
                return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
            a = min(max(math.floor(pair(high)), 0), rot_dim - 1)
            b = min(max(math.ceil(pair(low)), 0), rot_dim - 1)
            s = (0.0 if i <= a else 1.0) if a == b else min(max((i - a) / (b - a), 0.0), 1.0)
            t = t * (1 - s) + t / factor * s
            magnitude = 0.1 * math.log(factor) + 1
        got.append(t)
    return torch.tensor(got, dtype=torch.float64), magnitude


def pairs(rot_dim, interleaved):
    i = torch.arange(rot_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)


def rotate(x, positions, th, interleaved, magnitude=1.0, transpose=False):
    """x [..., D] turned by positions [...]; and the error bound of each value before
    its last rounding: the pair's magnitudes times what cosine and sine are off
    by, three fp32 roundings of products and sum, and the angle's own error (a
    fraction of a turn in 53 bits and one rounding, times the position)."""
    x = x.double()
    y, err = x.clone(), torch.zeros_like(x)
    a, b = pairs(2 * len(th), interleaved)
    ang = positions.double()[..., None] * th
    c, s = magnitude * torch.cos(ang), magnitude * torch.sin(ang)
    if transpose:
        s = -s
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    off = abs(magnitude) * (UCS + 4 * 2.0 ** -24 +
                            2 * math.pi * 2.0 ** -52 * positions.double().abs()[..., None])
    e = (x[..., a].abs() + x[..., b].abs()) * off
    err[..., a] = err[..., b] = e
    return y, err


def held_bf16(y, err):
    """Bound of a value rounded to bf16 (2^-126: subnormals count as zero)."""
    return err + UBF * (y.abs() + err) + 2.0 ** -126


def held_codes(y, err, fmt):
    """Bound of a row [..., D] that is held in 8 bits: half a step of its code
    (int8: of amax / 127; E4M3: 2^-4 of the value, and 2^-10 of amax / 448 where
    codes are subnormal), the value's and the largest value's own error, and a few
    fp32 roundings on the way there and back."""
    amax = y.abs().amax(-1, keepdim=True)
    e = err.amax(-1, keepdim=True)
    if fmt == "int8":
        half = 0.5 * (amax + e) / 127
    else:
        half = torch.maximum((y.abs() + e) * 2.0 ** -4, (amax + e) / 448 * 2.0 ** -10)
    return half * (1 + 2.0 ** -20) + 2 * e + 8 * 2.0 ** -24 * (y.abs() + e)


def tiles_values(pool, fmt):
    """What an 8-bit pool [NB, Hkv, 2112] stands for: [NB, Hkv, 16, D] in 64 bits."""
    codes = pool[..., :BLOCK * DIM].contiguous()
    codes = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().double()
    scales = pool[..., BLOCK * DIM:].contiguous().view(torch.float32).double()
    return codes.unflatten(-1, (BLOCK, DIM)) * scales[..., None]
