"""Rows of the root-mean-square norm whose squares or weighted values fp32 does not hold."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [64, 2056])
def test_rows_beyond_the_range_of_fp32(dtype, C):
    """Squares whose sum is no fp32 value: rstd is 0, and so are the outputs; 8-bit rows of them, and of products with
    the weight beyond the range, have a scale of NaN."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, C, generator=g)
    x[1] *= 2.0 ** 66
    x[2] *= 2.0 ** 40
    w = torch.ones(C)
    w[5], x[2, 5], x[0, 5] = 2.0 ** 110, 2.0 ** 40, 0.0
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    with gb.RMSNorm(C, dtype, max_N=3) as op:
        out, _, rstd = op.forward_train(x, w.cuda())
        q, scale, _ = op.forward_int8(x, w.cuda())
    assert rstd[1] == 0 and (out[1] == 0).all() and torch.isfinite(out[[0, 2]]).all() and (rstd[[0, 2]] > 0).all()
    assert torch.isfinite(scale[0]) and torch.isnan(scale[1:]).all() and (q[1:] == 0).all()
