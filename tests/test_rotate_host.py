"""Rotary positions without a GPU: the maps that the library fills in, against
their formulas, and the refusals of the C entry points and of the binding."""
import ctypes
import math

import pytest
import torch

from paged_kv_decode_18_gb300 import binding as B
from paged_kv_decode_18_gb300 import build as libbuild
from tests import rotate_ref as R

P = ctypes.c_void_p(0x10000)   # never dereferenced: every case fails host checks
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


SCALED = [
    dict(),
    dict(scaling="linear", factor=4.0),
    dict(scaling="base", factor=4.0),
    dict(base=500000.0, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0),
    dict(base=1e6, scaling="ramp", factor=4.0, original_len=32768, low=1.0, high=32.0),
    dict(base=1e6, scaling="ramp", factor=2.0, original_len=4096, low=3.0, high=3.0),
    # the whole ramp lies past the pairs, or before them
    dict(base=10.0, scaling="ramp", factor=2.0, original_len=1e6, low=1.0, high=32.0),
    dict(base=1e4, scaling="ramp", factor=2.0, original_len=6.0, low=1.0, high=32.0),
    dict(base=1.0),
]


@pytest.mark.parametrize("kw", SCALED, ids=lambda kw: kw.get("scaling", "none"))
@pytest.mark.parametrize("rot_dim", [2, 4, 30, 64, 128])
def test_angles_of_a_rotation(lib, rot_dim, kw):
    rot = B.make_rotation(rot_dim, interleaved=rot_dim == 64, **kw)
    th, magnitude = R.theta(rot_dim, **kw)
    assert rot.rot_dim == rot_dim and rot.interleaved == int(rot_dim == 64)
    assert rot.magnitude == pytest.approx(magnitude, rel=2.0 ** -24)
    for i in range(64):
        got = rot.turns[i] / 2.0 ** 64
        want = float(th[i]) / (2 * math.pi) % 1.0 if i < rot_dim // 2 else 0.0
        # a few roundings in 53 bits on either side (pow and log among them), and
        # the fraction cut off at its last place of 2^-64
        assert abs(got - want) <= 2.0 ** -48 * want + 2.0 ** -64, (i, got, want)


def test_angles_given_in_radians(lib):
    given = [1.0, -1.0, 0.0, 7.0, -1e-9, 2 * math.pi, 1e4]
    rot = B.make_rotation_from(torch.tensor(given, dtype=torch.float64), interleaved=True,
                               magnitude=1.5)
    assert (rot.rot_dim, rot.interleaved, rot.magnitude) == (14, 1, 1.5)
    for i, t in enumerate(given):
        want = t / (2 * math.pi)
        off = (rot.turns[i] / 2.0 ** 64 - want) % 1.0
        assert min(off, 1 - off) <= 2.0 ** -52 * max(1.0, abs(want))


def test_an_angle_times_a_position_is_exact(lib):
    # the integer product is the angle's fraction of a turn, at any position
    rot = B.make_rotation(128)
    for pos in (1, 77, 131071, 2 ** 30, -5, -2 ** 31):
        for i in (0, 1, 31, 63):
            got = (rot.turns[i] * pos) % 2 ** 64 / 2.0 ** 64
            want = pos * float(R.theta(128)[0][i]) / (2 * math.pi)
            off = (got - want) % 1.0
            assert min(off, 1 - off) <= abs(pos) * 2.0 ** -51


def test_rotation_refusals(lib):
    def init(rot_dim=128, base=1e4, kind=0, factor=1.0, n=8192.0, low=1.0, high=4.0, null=False):
        rot = B.pa_rotation()
        return lib.pa_rotation_init(None if null else ctypes.byref(rot), rot_dim, 0, base, kind,
                                    factor, n, low, high)
    nan, inf = float("nan"), float("inf")
    assert init() == B.PA_OK
    for bad in (dict(null=True), dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130),
                dict(rot_dim=-2), dict(base=0.0), dict(base=-1.0), dict(base=nan), dict(base=inf),
                dict(kind=-1), dict(kind=5), dict(kind=1, factor=0.0), dict(kind=1, factor=nan),
                dict(kind=2, factor=inf), dict(kind=3, n=0.0), dict(kind=3, low=4.0),
                dict(kind=3, low=0.0), dict(kind=3, high=nan), dict(kind=4, n=inf),
                dict(kind=4, low=5.0), dict(kind=4, base=1.0), dict(kind=4, high=inf)):
        assert init(**bad) == B.PA_ERR_ARG, bad
    assert init(kind=4, low=4.0) == B.PA_OK
    one = (ctypes.c_double * 64)(*[1.0] * 64)
    rot = B.pa_rotation()
    ref = ctypes.byref(rot)
    assert lib.pa_rotation_set(ref, 128, 0, one, 1.0) == B.PA_OK
    assert lib.pa_rotation_set(None, 128, 0, one, 1.0) == B.PA_ERR_ARG
    assert lib.pa_rotation_set(ref, 128, 0, None, 1.0) == B.PA_ERR_ARG
    assert lib.pa_rotation_set(ref, 0, 0, one, 1.0) == B.PA_ERR_ARG
    assert lib.pa_rotation_set(ref, 128, 0, one, nan) == B.PA_ERR_ARG
    one[63] = inf
    assert lib.pa_rotation_set(ref, 128, 0, one, 1.0) == B.PA_ERR_ARG
    assert lib.pa_rotation_set(ref, 126, 0, one, 1.0) == B.PA_OK
    with pytest.raises(ValueError, match="scaling"):
        B.make_rotation(128, scaling="bend")
    with pytest.raises(B.PAError):
        B.make_rotation(127)
    with pytest.raises(B.PAError):
        B.make_rotation_from([])


def view(data=0x10000, ts=2048, hs=128):
    return ctypes.byref(B.pa_row_view(data, ts, hs))


BAD_VIEWS = [dict(data=None), dict(data=0x10008), dict(ts=2044), dict(hs=124), dict(ts=-2048),
             dict(hs=-128), dict(ts=1 << 60), dict(hs=1 << 60)]
LYING_OVER = [dict(hs=0), dict(hs=64), dict(ts=0), dict(ts=1920), dict(ts=128, hs=128),
              dict(ts=128, hs=256)]


def test_rotate_refusals(lib):
    def call(x=None, y=None, pos=P, T=4, H=16, D=128, rot=None, null_rot=False):
        rot = rot or B.make_rotation(128)
        return lib.pa_rotate(x or view(), pos, T, H, D, None if null_rot else ctypes.byref(rot), 0,
                             y or view(0x90000), None)
    assert call(D=64) == B.PA_ERR_UNSUPPORTED
    assert call(H=1 << 25) == B.PA_ERR_UNSUPPORTED or call(H=1 << 25) == B.PA_ERR_ARG
    assert call(T=1 << 40, x=view(ts=8), y=view(0x90000, ts=2048)) in (B.PA_ERR_UNSUPPORTED,
                                                                       B.PA_ERR_ARG)
    assert call(D=0) == B.PA_ERR_ARG
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(H=-1) == B.PA_ERR_ARG
    assert call(pos=None) == B.PA_ERR_ARG
    assert call(pos=ODD) == B.PA_ERR_ARG
    assert call(null_rot=True) == B.PA_ERR_ARG
    for kw in BAD_VIEWS:
        assert call(x=view(**kw)) == B.PA_ERR_ARG, kw
        assert call(y=view(**kw)) == B.PA_ERR_ARG, kw
    for kw in LYING_OVER:
        assert call(y=view(**{"data": 0x90000, **kw})) == B.PA_ERR_ARG, kw
    assert call(x=view(), y=view(ts=4096)) == B.PA_ERR_ARG   # in place with other strides
    for field, value in (("rot_dim", 0), ("rot_dim", 3), ("rot_dim", 256), ("interleaved", 2),
                         ("magnitude", float("inf"))):
        rot = B.make_rotation(128)
        setattr(rot, field, value)
        assert call(rot=rot) == B.PA_ERR_ARG, field
    assert call(T=0, pos=None) == B.PA_OK
    assert call(H=0, pos=None) == B.PA_OK


def shape(**kw):
    base = dict(num_seqs=4, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16,
                max_blocks_per_seq=24, num_blocks=128)
    base.update(kw)
    return B.make_shape(**base)


def test_rotate_and_cache_refusals(lib):
    def call(q=True, k=None, v=None, qo=True, pos=P, slots=P, T=4, kc=P, vc=P, fmt=0, sh=None,
             rot=None):
        rot = rot or B.make_rotation(128)
        q = view() if q is True else q
        qo = view(0x90000) if qo is True else qo
        return lib.pa_rotate_and_cache(q, k or view(0x20000), v or view(0x30000), pos, slots, T,
                                       ctypes.byref(rot), qo, kc, vc, fmt,
                                       ctypes.byref(sh or shape()), None)
    assert call(sh=shape(head_dim=64)) == B.PA_ERR_UNSUPPORTED
    assert call(sh=shape(num_q_heads=12)) == B.PA_ERR_ARG
    assert call(fmt=3) == B.PA_ERR_ARG
    assert call(fmt=-1) == B.PA_ERR_ARG
    assert call(T=-1) == B.PA_ERR_ARG
    assert call(q=None) == B.PA_ERR_ARG
    assert call(qo=None) == B.PA_ERR_ARG
    assert call(pos=None) == B.PA_ERR_ARG
    assert call(slots=None) == B.PA_ERR_ARG
    assert call(slots=ctypes.c_void_p(0x10004)) == B.PA_ERR_ARG
    assert call(kc=None) == B.PA_ERR_ARG
    assert call(vc=ctypes.c_void_p(0x10008)) == B.PA_ERR_ARG
    assert call(qo=view(0x10000, ts=4096)) == B.PA_ERR_ARG
    for kw in BAD_VIEWS:
        assert call(k=view(**kw)) == B.PA_ERR_ARG, kw
        assert call(v=view(**kw)) == B.PA_ERR_ARG, kw
        assert call(q=view(**kw)) == B.PA_ERR_ARG, kw
    rot = B.make_rotation(128)
    rot.rot_dim = 5
    assert call(rot=rot) == B.PA_ERR_ARG
    assert call(T=0, pos=None, slots=None, kc=None) == B.PA_OK
    assert call(T=0, q=None, qo=None) == B.PA_OK


def test_rotate_cached_refusals(lib):
    def call(kc=P, fmt=0, tables=P, lens=P, shifts=P, first=0, kept=None, n=0, sh=None):
        rot = B.make_rotation(128)
        return lib.pa_rotate_cached(kc, fmt, tables, lens, shifts, first, kept, n,
                                    ctypes.byref(rot), ctypes.byref(sh or shape()), None)
    assert call(sh=shape(block_size=32)) == B.PA_ERR_UNSUPPORTED
    assert call(fmt=7) == B.PA_ERR_ARG
    assert call(shifts=None) == B.PA_ERR_ARG
    assert call(kept=P) == B.PA_ERR_ARG
    assert call(first=-1) == B.PA_ERR_ARG
    assert call(n=5) == B.PA_ERR_ARG
    assert call(shifts=None, kept=P, n=-1) == B.PA_ERR_ARG
    assert call(shifts=None, kept=P, n=5, first=1) == B.PA_ERR_ARG
    assert call(kc=None) == B.PA_ERR_ARG
    assert call(kc=ODD) == B.PA_ERR_ARG
    assert call(tables=None) == B.PA_ERR_ARG
    assert call(lens=ODD) == B.PA_ERR_ARG
    assert call(shifts=ODD) == B.PA_ERR_ARG
    assert call(sh=shape(num_seqs=0)) == B.PA_OK
    assert call(sh=shape(max_blocks_per_seq=0)) == B.PA_OK


def test_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros((4, 16, 128), dtype=torch.bfloat16)
    pos = torch.zeros((4,), dtype=torch.int32)
    rot = B.pa_rotation(128, 0, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        B.prepare_rotate(x, pos, rot, x)
    with pytest.raises(ValueError, match="required"):
        B.prepare_rotate(None, pos, rot, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.prepare_rotate_and_cache(x, x, pos, pos, rot, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.prepare_rotate_cached(torch.zeros((2, 8, 16, 128), dtype=torch.bfloat16), pos[None], pos,
                                rot, shifts=pos)
