"""A kernel whose launch overlaps the one before it reads that kernel's results by plain loads: the read-only data path is
defined only for memory that nobody writes during a kernel's life, which begins before those results are there."""
import os
import re

import pytest

import tiled_distributed_attention_gb300 as m

CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")


def code_of(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


OVERLAPPED = sorted(n for n in os.listdir(CSRC) if n.endswith(".cu") and "wait_for_kernel_before()" in code_of(n))


def test_the_overlapped_files_are_found():
    assert {"rope.cu", "diff_aux.cu", "diff_fwd_tc.cu", "diff_bwd_tc.cu", "diff_bwd_tc32.cu", "diff_decode.cu",
            "tile_fwd_tc32.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("name", OVERLAPPED)
def test_no_read_only_loads(name):
    left = [line.strip() for line in code_of(name).splitlines()
            if re.search(r"__ldg\s*\(|ld\.global\.nc", line)
            and "prm.kv_list" not in line]  # of a plan's tables, which no kernel writes
    assert not left, left
    # nor by the compiler's choice: a kernel's pointers are not marked as unaliased
    for kernel in re.findall(r"__global__[^{;]*\{.*?\n\}", code_of(name), flags=re.S):
        if "wait_for_kernel_before()" in kernel:
            assert "__restrict__" not in kernel.split("{")[0]
