"""The bound of dweight notices one row left out of it, or taken twice."""
import pytest
import torch

import linear_oracle as no
import rms_depth as rd

SIZES = [(9001, 72), (3001, 1032), (5003, 2560), (2055, 4096), (70001, 8)]


@pytest.mark.parametrize("N,C", SIZES)
def test_a_row_missing_or_twice(N, C):
    g = torch.Generator().manual_seed(1)
    h, d = torch.randn(N, C, generator=g), torch.randn(N, C, generator=g)
    value, bound = rd.dweight(h, d, 256)
    no.check("rounded", value.float(), value, bound)
    rstd = no.rms(h, None)[2]
    for row in (0, 1, N // 2, N - 1):
        term = d[row].double() * h[row].double() * rstd[row]
        for wrong in (value - term, value + term):
            with pytest.raises(AssertionError):
                no.check("planted", wrong.float(), value, bound)


def test_depths():
    assert rd.blocks(72, 9001, 256) == 1024 and rd.depth(72, 9001, 256) == 3 + 4 + 32 + 5
    assert rd.blocks(1032, 3001, 256) == 1024 and rd.depth(1032, 3001, 256) == 3 + 32 + 5
    assert rd.blocks(4096, 2055, 256) == 512 and rd.depth(4096, 2055, 256) == 5 + 16 + 5
