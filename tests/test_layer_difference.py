"""The difference test of the diagonal recurrence's gradient, pinned on the CPU: its tolerance is far
below what it measures, for every input."""
import pytest

import layer_difference as ld
import layer_oracle as lo


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("name", ld.INPUTS)
def test_a_gradient_two_percent_off_is_caught(name, gate, reverse):
    x = ld.inputs(94, gate)
    _, _, step, difference, tol, _ = ld.along_gradient(x, name, reverse)
    grad = lo.glr_grad(x["v"], x["beta"], x["decay"], x["dout"], x["state"], x["dstate"], reverse)[ld.INPUTS[name]][0]
    right = (grad * step).sum().item()
    assert abs(right - difference) <= tol < 0.01 * abs(right)
    for wrong in (0.0, 0.98, 1.02, -1.0):
        assert abs(wrong * right - difference) > tol
