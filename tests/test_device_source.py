"""Rules that the kernels' sources keep, checked on their text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_decode_18_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def code(path):
    """The file without its comments."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", " ", text, flags=re.S)


def enclosed(text, at, pair):
    """The text from the opening bracket at `at` to its partner."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("unbalanced brackets")


def kernels(text):
    """(name, parameters, body) of the kernels that a text defines."""
    for m in re.finditer(r"__global__ void(?: __launch_bounds__)?", text):
        at = m.end()
        if m.group(0).endswith("__launch_bounds__"):
            at += len(enclosed(text, at, "()"))
        name = re.compile(r"\s*(\w+)").match(text, at)
        params = enclosed(text, name.end(), "()")
        brace = text.index("{", name.end() + len(params))
        yield name.group(1), params, enclosed(text, brace, "{}")


def test_every_kernel_is_found():
    names = [k[0] for f in FILES for k in kernels(code(f))]
    assert len(names) == sum(len(re.findall(r"\b__global__\b", code(f))) for f in FILES)
    assert {"tree_mask_kernel", "evict_kernel", "weights_tc_kernel"} <= set(names)


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_what_an_earlier_grid_may_write_is_read_by_ordinary_loads(path):
    # A kernel that starts before the grid ahead of it has ended (griddepcontrol)
    # runs while its inputs are still being written. The non-coherent path is
    # for data that nobody writes while the kernel runs: no intrinsic that takes it, and
    # no pointer that says so to the compiler.
    text = code(path)
    assert "__ldg(" not in text and "ld.global.nc" not in text
    for name, params, body in kernels(text):
        if "griddepcontrol.wait" in body:
            told = re.findall(r"const\s+[\w:]+\s*\*\s*__restrict__\s+(\w+)", params)
            assert not told, (name, told)
