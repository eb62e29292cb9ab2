"""The order of LDS accesses between the waves of the 8-bit product's tiles, from the assembly: a wave's reads of a stage
are over before the barrier behind which other waves' copies write it anew.  A wrong order shows as a wrong sum only
where a copy is quicker than a read, so values do not test it."""
import os
import re

import pytest

import assembly
from gated_deltanet_recurrence_gdn_amd import build

FORMS = pytest.mark.parametrize("side,out", [(256, "fp32"), (256, "bf16"), (128, "fp32"), (128, "bf16")])


def tile_kernel(side, out):
    found = {n: x for n, x in assembly.kernels("gdn_matmul.hip").items() if "matmul_tile_kernel" in n}
    assert len(found) == 4
    (lines,) = (x for n, x in found.items() if f"ILi{side}ELi{side}E" in n and f"ELb{int(out == 'fp32')}E" in n)
    return lines


@FORMS
def test_reads_of_a_stage_end_before_the_barrier(side, out):
    lines = tile_kernel(side, out)
    barriers = [i for i, x in enumerate(lines) if x == "s_barrier"]
    assert len(barriers) == 2  # a loop over pairs of stages
    for i in barriers:
        j = i
        while not lines[j].startswith("s_waitcnt"):
            j -= 1
            assert not re.match(r"ds_|buffer_|global_|s_c?branch|\.LBB", lines[j]), f"{lines[j]} between the wait and the barrier"
        assert "lgkmcnt(0)" in lines[j], f"reads of LDS may be under way at the barrier behind {lines[j]!r}"
        assert "vmcnt(" in lines[j]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_the_load_that_touches_lines_is_the_youngest(out):
    """The wide form waits for all loads but one before a barrier: the one left under way must be the load of four bytes
    whose data nobody reads, in the loop and before it, and the source must say so to the scheduler."""
    lines = tile_kernel(256, out)
    for i in (i for i, x in enumerate(lines) if x == "s_barrier"):
        behind = next(j for j in range(i - 1, 0, -1) if lines[j].startswith("s_waitcnt"))
        assert re.search(r"vmcnt\(1\)", lines[behind])
        loads = [x.split()[0] for x in lines[:i] if re.match(r"(buffer|global)_load", x)]
        assert loads[-1] == "buffer_load_dword" and loads[-2] == "buffer_load_dwordx4"
    with open(os.path.join(build.CSRC, "gdn_matmul.hip")) as f:
        body = re.search(r"const auto touch = .*?\n    };", f.read(), re.S)[0]
    first = body.index("sched_barrier(0)")
    assert first < body.index("load4_to_lds") < body.index("sched_barrier(0)", first + 1)
