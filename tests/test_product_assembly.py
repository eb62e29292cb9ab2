"""The order of LDS accesses between the waves of the 8-bit product's tiles, from the assembly: a wave's reads of a stage
are over before the barrier behind which other waves' copies write it anew.  A wrong order shows as a wrong sum only
where a copy is quicker than a read, so values do not test it."""
import re

import pytest

import assembly

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
