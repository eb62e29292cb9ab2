"""The diagonal recurrence's gradient on the GPU against differences of its own forward pass, along
the gradient of each input."""
import pytest

import layer_difference as ld
import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("name", ld.INPUTS)
def test_gradient_is_the_difference(name, gate, reverse):
    x = ld.inputs(94, gate)
    hi, low, step, difference, tol, forward = ld.along_gradient(x, name, reverse)
    B, T, H, d = x["v"].shape
    with gb.GLR(B, H, d, "fp32", max_T=T, gate=gate, reverse=reverse) as g:
        def loss(z):
            c = lo.cuda(z)
            out, st = g.forward(c["v"], c["beta"], c["decay"], state_in=c["state"])
            return ld.loss(x, out.cpu(), st.cpu())
        got = loss(hi) - loss(low)
        c = lo.cuda(x)
        _, _, saved = g.forward_train(c["v"], c["beta"], c["decay"], state_in=c["state"])
        grads = dict(zip(ld.INPUTS, g.backward(c["v"], c["beta"], c["decay"], saved, c["dout"], c["dstate"])))
    assert abs(got - difference) <= forward
    assert abs((grads[name].cpu().double() * step).sum().item() - got) <= tol
