"""8-bit rows next to the middle of two levels, closer than 64-bit quotients tell."""
from fractions import Fraction

import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

# h and weight of the largest product of a row, and of one whose level is within 2^-47 of a middle: 24 bits each, found by
# searching factors of ((2 k + 1) top +- 2) / 254.  127 h w / top in 64 bits has the middle itself, or falls on its other side.
NEAR = [
    (9250540, 11945774, 14287697, 7216619),
    (11164987, 8727123, 13298137, 7125277),
    (16010557, 12086171, 16289974, 8651926),
    (8721585, 10026255, 11866363, 4554938),
    (16705482, 8754861, 12058042, 10171321),
    (13430267, 11209314, 14921453, 8857756),
    (9642167, 15840677, 15786815, 6056438),
    (8951036, 10906356, 16710481, 5451031),
    (10132671, 9914189, 9072923, 7105388),
    (13514411, 9152457, 15991823, 6364282),
    (15169623, 15449921, 11495116, 10354847),
    (11510141, 9661657, 11395981, 9028481),
]


def level(p, top):
    """The nearest whole number to 127 p / top, ties to even."""
    return round(Fraction(127) * p / top)  # of a Fraction: exact


def test_quotients_in_64_bits_miss_these():
    for a, b, c, d in NEAR:
        assert round(127.0 * float(c * d) / float(a * b)) != level(c * d, a * b)


@pytest.mark.parametrize("C", [16, 1024, 1096, 8192])
@pytest.mark.parametrize("power", [0, -24, -60, 20])
def test_levels_next_to_a_middle(C, power):
    with gb.RMSNorm(C, "fp32", max_N=4) as op:
        for i, (a, b, c, d) in enumerate(NEAR):
            at, to = (3 * i) % C, (C - 1 - 5 * i) % C
            h, w = torch.zeros(4, C, dtype=torch.float64), torch.ones(C, dtype=torch.float64)
            w[at], w[to] = b, d
            # the top, and the near one on both sides of zero; both at a time swapped in sign
            h[0, at], h[0, to] = a, c
            h[1, at], h[1, to] = a, -c
            h[2, at], h[2, to] = -a, c
            h[3, at], h[3, to] = -a, -c
            q, _, _ = op.forward_int8((h * 2.0 ** (power - 24)).float().cuda(), (w * 2.0 ** -24).float().cuda())
            k = level(c * d, a * b)
            assert q[:, to].tolist() == [k, -k, k, -k], (i, k)
            assert q[:, at].tolist() == [127, 127, -127, -127]
