"""The state's gradient written over the one that came in, in every form of the cut, whatever else is wanted."""
import pytest
import torch

import linear_cuts as lc
import linear_oracle as no
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dlog", "dstate")


@pytest.mark.parametrize("dtype,d", [("bf16", 16), ("fp32", 16), ("bf16", 128)])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("H,T", [(2, 1), (3, 50), (300, 192), (2, 200), (60, 683)])  # one chunk; one segment; segments of one chunk, of three
def test_gradient_of_the_state(H, T, dtype, d, reverse):
    n = lc.grad_cut(H, lc.up(T, 64), torch.cuda.get_device_properties(0).multi_processor_count)[1]
    assert (n == 1) == ((H, T) in ((2, 1), (3, 50), (300, 192)))
    x = no.linear_inputs(1, 1, T, H, d, d, dtype)
    c = {m: y.cuda() for m, y in x.items()}
    with gb.LinearAttention(1, H, d, d, dtype, max_T=T, reverse=reverse, train=True) as op:
        want = op.backward(c["q"], c["k"], c["v"], c["decay"], c["dout"], state_in=c["state"], dstate_out=c["dstate"])
        s = torch.cuda.current_stream().cuda_stream
        rows = [v for m in ("q", "k", "v") for v in (c[m], H * d, T * H * d)]
        for skip in (None, 0, 1, 2, 3, (0, 1, 2), (0, 1, 2, 3)):
            skip = skip if isinstance(skip, tuple) else (skip,)
            bufs = [torch.full_like(y, 5) for y in want[:4]] + [c["dstate"].clone()]
            args = [None if i in skip else b for i, b in enumerate(bufs)]
            st = gb.gdn_linear_backward(op.h, *rows, c["decay"], c["state"], c["dout"], bufs[4], *args, T, s)
            assert st == gb.GDN_OK, gb.gdn_last_error(op.h)
            torch.cuda.synchronize()
            for i, m in enumerate(NAMES):
                assert torch.equal(bufs[i], torch.full_like(want[i], 5) if i in skip else want[i]), (skip, m)
