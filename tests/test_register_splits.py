"""A kernel that hands registers between its warpgroups is launched only where the launch has them: a warpgroup that raises
its registers beyond that waits for ever."""
import os
import re

import pytest

import tiled_distributed_attention_gb300 as m

CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")
SPLIT = sorted(n for n in os.listdir(CSRC) if n.endswith(".cu") and "regs_inc<" in open(os.path.join(CSRC, n)).read())


@pytest.mark.parametrize("name", SPLIT)
def test_launcher_checks_the_split(name):
    src = open(os.path.join(CSRC, name)).read()
    used = set(re.findall(r"regs_(?:inc|dec)<(\w+)>", src))
    check = re.search(r"fa\.numRegs \* NUM_THREADS < ([^)]*)\)", src)
    assert check and all(n in check.group(1) for n in used), used
    # and as the constants stand, it fits 168 (three warps of a sub-partition) or 128 (four) registers a thread
    value = {n: int(v) for n, v in re.findall(r"(\w+_REGS) = (\d+)", src)}
    threads = int(re.search(r"NUM_THREADS = (\d+);", src).group(1))
    need = eval(check.group(1), {}, value)
    assert need <= threads * {384: 168, 512: 128}[threads]


def test_all_are_found():
    assert {"tile_fwd_tc.cu", "tile_bwd_tc.cu", "diff_fwd_tc.cu", "diff_bwd_tc.cu", "diff_bwd_tc32.cu"} <= set(SPLIT)
