"""The root-mean-square norm's gradient where waves and blocks walk several rows, the last round of them not full:
dweight within the depth of its sums, dx of every row, and the same bits every time."""
import pytest
import torch

import linear_oracle as no
import rms_depth as rd
from gated_deltanet_recurrence_gdn_amd import binding as gb
from test_rms_depth import SIZES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("N,C", SIZES)
def test_rows_after_rows(N, C, weight, dtype):
    g = torch.Generator().manual_seed(1)
    h, d, ds = (torch.randn(N, C, generator=g).to(no.DT[dtype]) for _ in range(3))
    w = 1 + 0.2 * torch.randn(C, generator=g) if weight else None
    ncu = torch.cuda.get_device_properties(0).multi_processor_count
    n = rd.blocks(C, N, ncu)
    assert N > (n if C > 1024 else 4 * n) and N % (n if C > 1024 else 4 * n)
    with gb.RMSNorm(C, dtype, max_N=N) as op:
        hc, dc, dsc, wc = h.cuda(), d.cuda(), ds.cuda(), None if w is None else w.cuda()
        _, _, rstd = op.forward_train(hc, wc)
        dx, dw = op.backward(hc, wc, rstd, dc, dsum=dsc)
        dx2, dw2 = op.backward(hc, wc, rstd, dc, dsum=dsc)
        assert torch.equal(dx, dx2)
        no.check("dx", dx, *no.rms_grad(h, w, d, ds)["dx"])
        if weight:
            assert torch.equal(dw, dw2)
            no.check("dweight", dw, *rd.dweight(h, d, ncu))
        else:
            # of a weight that is all ones and not given, its gradient still is wanted by a C caller
            raw = torch.empty(C, device="cuda")
            st = gb.gdn_rms_norm_backward(op.h, hc, None, rstd, dc, dsc, None, raw, N, torch.cuda.current_stream().cuda_stream)
            assert st == gb.GDN_OK
            no.check("dweight", raw, *rd.dweight(h, d, ncu))
