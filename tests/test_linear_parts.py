"""The model of operands in bf16 parts against the definition: exact with parts enough, and told apart with two."""
import pytest

import linear_oracle as no
import linear_parts as lp


@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64)])
def test_parts(dk, dv):
    x = no.linear_inputs(1, 1, 192, 3, dk, dv)
    ref = no.linear(x)
    for name, y in lp.linear(x, 8).items():  # (parts of what fp32 holds of an operand: 2^-25 at most left out)
        assert no.rel_l2(y, ref[name][0]) < 1e-7, name
    two, three = lp.linear(x, 2), lp.linear(x, 3)
    for name in two:
        e2, e3 = no.rel_l2(two[name], ref[name][0]), no.rel_l2(three[name], ref[name][0])
        print(name, e2, e3)
        assert e2 > 1e-6 and e3 < e2 / 16, name
