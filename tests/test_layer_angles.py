"""The documented bound of the rotary angle, on the CPU: the kernel's formula for a pair's frequency
against fifty digits.  An angle is off by at most 2^-50 of a radian per unit of position; relative
to the angle itself no such bound holds, the exponent being rounded before the power is taken."""
from decimal import Decimal
import math

import pytest

from layer_angles import PI, frequencies


@pytest.mark.parametrize("theta", [1.5, 100.0, 1e4, 1e6, 1e8, 1e100, 1e300])
def test_frequency_error(theta):
    most = 0.0
    for n in (2, 6, 16, 42, 44, 128, 170, 510, 512):
        for i, exact in enumerate(frequencies(n, theta)):
            turns = 2.0 ** (-2.0 * i / n * math.log2(theta)) * 0.15915494309189533577
            # the product with the position is off by half a step more, exp2 on the device by a step of its own
            most = max(most, float(abs(Decimal(turns) * 2 * PI - exact) + exact * Decimal(3 * 2.0 ** -53)))
    assert most <= 2.0 ** -50


def test_closed_forms():
    assert frequencies(4, 16.0) == pytest.approx([1, Decimal("0.25")])
