"""What leaves in fp32 on the bf16 path goes through operands in three bf16 parts: states, their gradients and the decay's
gradient are less than half as far off as two parts alone would leave them (tests/linear_parts.py), every other step
exact.  With three parts that share is 1/64; fp32 steps add some u, a tenth to a third of it."""
import pytest
import torch

import linear_oracle as no
import linear_parts as lp
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 32), (32, 64), (64, 32), (64, 64), (64, 128), (128, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("H", [3, 300])  # segments of one chunk, and a call in one piece
def test_three_parts(H, dk, dv, dtype):
    x = no.linear_inputs(1, 1, 192, H, dk, dv, dtype)
    c = {n: y.cuda() for n, y in x.items()}
    with gb.LinearAttention(1, H, dk, dv, dtype, max_T=192, train=True) as op:
        _, state = op.forward(c["q"], c["k"], c["v"], c["decay"], state_in=c["state"])
        *_, dlog, dstate = op.backward(c["q"], c["k"], c["v"], c["decay"], c["dout"], state_in=c["state"], dstate_out=c["dstate"])
    some = list(range(0, H, 1 if H < 10 else 60))
    pick = lambda n, y: y[:, some] if "state" in n else y[:, :, some]  # noqa: E731
    y = {n: pick(n, t) for n, t in x.items()}
    ref, two = no.linear(y, dtype=dtype), lp.linear(y, 2)
    for name, got in (("state", state), ("dstate", dstate), ("dlog", dlog)):
        e, e2 = no.rel_l2(pick(name, got), ref[name][0]), no.rel_l2(two[name], ref[name][0])
        print(f"{name}: {e:.2e}, two parts {e2:.2e}")
        assert e < e2 / 2, f"{name}: {e:.2e}, two parts alone {e2:.2e}"
