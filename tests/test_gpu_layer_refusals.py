"""Refusals of the torch wrappers that need tensors on a GPU; no kernel is launched."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

SHAPES = [(2, 0, 3, 16), (0, 5, 3, 16), (2, 5, 0, 16)]


@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_of_nothing(shape):
    x = torch.empty(shape, device="cuda")
    pos = torch.zeros((shape[1], 3), dtype=torch.int32, device="cuda")
    assert gb.rotary(x, (4, 4, 4), grid=(1, 1)).shape == shape
    assert gb.rotary(x, (4, 4, 4), positions=pos).shape == shape
    assert gb.rotary(x, (4, 4, 4), grid=(2, 3), out=x) is x


@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_of_nothing_is_checked_like_any_other(shape):
    x = torch.empty(shape, device="cuda")
    with pytest.raises(ValueError, match="positions or grid"):
        gb.rotary(x, (4, 4, 4))
    with pytest.raises(ValueError, match="positions"):
        gb.rotary(x, (4, 4, 4), positions=torch.zeros((shape[1], 3), device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        gb.rotary(x, (4, 4, 4), positions=torch.zeros((shape[1] + 1, 3), dtype=torch.int32, device="cuda"))
    for how in (dict(axis_dims=(3, 4, 4)), dict(axis_dims=(8, 8, 2)), dict(axis_dims=(-2, 4, 4)), dict(theta=0.5),
                dict(theta=float("nan")), dict(grid=(0, 5)), dict(first_token=-1)):
        with pytest.raises(gb.GDNError):
            gb.rotary(x, **{"axis_dims": (4, 4, 4), "grid": (1, 1), **how})
    with pytest.raises(gb.GDNError):
        gb.rotary(torch.empty((2, 0, 3, 12), device="cuda"), (4, 4, 4), grid=(1, 1))
