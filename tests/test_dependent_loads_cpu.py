"""Kernels that start before the kernel ahead of them has ended (they call
griddepcontrol.wait) must not read what that kernel writes through the read-only
path: it asks for data that stays as it is for the whole life of the kernel, and
allows the compiler to move the load above the wait.  The sources are checked:
such a kernel takes no `const T* __restrict__` but the compressed weights, and
the files whose kernels are all of this kind hold no __ldg."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prng_seeded_decompress_b200", "csrc")
#: Records and exponents: nothing writes them while a product runs.
WEIGHTS = {"rec", "eplane"}


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def closing(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise AssertionError("unbalanced")


def kernels(text):
    """(name, parameters, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        at = m.end()
        while True:  # over the launch bounds, to the name and its parameters
            k = re.compile(r"(\w+)\s*\(").search(text, at)
            end = closing(text, k.end() - 1, "()")
            if k.group(1) != "__launch_bounds__":
                break
            at = end
        rest = text[end + 1:].lstrip()
        if rest.startswith("{"):
            start = text.index("{", end)
            yield k.group(1), text[k.end():end], text[start:closing(text, start, "{}")]


def waits(body):
    return "griddepcontrol.wait" in body or "grid_wait()" in body


BETWEEN = ["adapters.cu", "block_norm.cu"]
PRODUCTS = ["gemv.cu", "gemv_amort.cu", "gemm_cc.cu", "gemm_tc.cu"]


@pytest.mark.parametrize("name", BETWEEN + PRODUCTS)
def test_nothing_that_may_still_be_written_is_read_only(name):
    found = [k for k in kernels(source(name)) if waits(k[2])]
    assert found
    for kernel, params, _ in found:
        for param in re.findall(r"const\s[^,]*?\*\s*__restrict__\s*(\w+)", params):
            assert param in WEIGHTS, f"{kernel}: {param}"


@pytest.mark.parametrize("name", BETWEEN)
def test_files_of_such_kernels_alone_hold_no_read_only_loads(name):
    text = source(name)
    found = list(kernels(text))
    assert len(found) >= 5 and all(waits(body) for _, _, body in found)
    assert "__ldg" not in text and "ld.global.nc" not in text
