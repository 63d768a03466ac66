"""The plan's costs of the tcgen05 weights kernel, compiled for the host."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_decode_18_gb300", "csrc")


@pytest.fixture(scope="module")
def cost(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cc", d / "plan.so"
    src.write_text('#include "pa_weights_plan.h"\n'
                   'extern "C" int cost(int nt, int c, int lq, int qtb, int hkv, int s) {\n'
                   '  return pa::window_cost(nt, c, lq, qtb, hkv, s);\n}\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-ftrapv", "-I", CSRC,
                    "-o", str(lib), str(src)], check=True)
    return ctypes.CDLL(str(lib)).cost


def by_hand(c, lq, qtb, hkv):
    """One for each (key tile, head) and one for each query tile with a token that
    sees a key of it."""
    n = 0
    for lo in range(0, c, 128):
        tiles = {j // qtb for j in range(lq) if lo <= c - lq + j}
        n += 1 + (len(tiles) if lq > qtb else -(-lq // qtb))
    return n * hkv


def test_costs_are_the_tiles_of_a_window(cost):
    rng = random.Random(1)
    for _ in range(60):
        c = rng.randint(1, 1500)
        lq, qtb, hkv = rng.randint(0, c), rng.choice([1, 5, 16, 42, 64, 128]), rng.choice([1, 2, 8])
        assert cost(-(-c // 128), c, lq, qtb, hkv, 3) == by_hand(c, lq, qtb, hkv)


@pytest.mark.parametrize("c,qtb,hkv,seqs", [(1 << 20, 17, 8, 1), (1 << 20, 1, 64, 5),
                                            (1 << 22, 3, 8, 256), ((1 << 22) - 5, 1, 1, 4000)])
def test_windows_longer_than_announced_keep_the_sum_in_32_bits(cost, c, qtb, hkv, seqs):
    nt = -(-c // 128)
    one = cost(nt, c, c, qtb, hkv, seqs)
    nq, exact = -(-c // qtb), 0
    for kt in range(nt):
        exact += 1 + nq - kt * 128 // qtb
    assert exact * hkv >= 1 << 30 or seqs > 1
    assert one == min(exact * hkv, (1 << 30) // seqs)
    assert 0 < one * seqs <= 1 << 30
