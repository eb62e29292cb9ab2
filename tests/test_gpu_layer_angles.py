"""Rotary positions on the GPU at the ends of the position range, within the documented bound of the
angle: 2^-50 of a radian per unit of position, against angles of fifty digits."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb
from layer_angles import frequencies, turn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("theta", [100.0, 1e4, 1e6, 1e8, 1e300])
@pytest.mark.parametrize("n", [44, 128])
def test_far_positions(n, theta):
    places = [0, 1, -1, 4095, 2**24 + 1, 2**26, 2**31 - 1, -2**31, 1234567891]
    x = torch.zeros((1, len(places), 1, 128), device="cuda")
    x[..., :n:2] = 1.0
    pos = torch.tensor([[p, 0, 0] for p in places], dtype=torch.int32, device="cuda")
    y = gb.rotary(x, (n, 0, 0), theta=theta, positions=pos)[..., :n]
    f = frequencies(n, theta)
    ref = torch.tensor([[c for g in f for c in turn(p, g)] for p in places], dtype=torch.float64).reshape(1, len(places), 1, n)
    # cosine and sine of an fp32 fraction of a turn: 8 u, as in layer_oracle.rotary
    bound = (8 * lo.U + 2.0 ** -50 * torch.tensor(places, dtype=torch.float64).abs())[None, :, None, None].expand_as(ref)
    lo.check("far positions", y, ref, bound)
