"""Calls of the operators around the recurrence that are refused for their extents or their
arguments together, without a GPU."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

A = [(1 << 40) + i * (1 << 30) for i in range(8)]


@pytest.mark.parametrize("C,N,S", [(1024, 1 << 24, 1 << 30), (8192, 1 << 21, 1 << 30), (8192, 1 << 24, 1 << 28),
                                   (1024, (1 << 24) - 1, 1 << 30), (64, 1 << 24, 1 << 30)])
def test_group_norm_extents_beyond_64_bits(C, N, S):
    """N, S and C within their own limits whose product (in bytes) is not: a wrapped size would let NULL and
    overlapping tensors through."""
    st, h = gb.gdn_group_norm_create(-1, C, 4, gb.GDN_F32, gb.GDN_ACT_SILU, 1e-5, 1 << 24)
    assert st == gb.GDN_OK
    try:
        for x, out in ((A[0], A[3]), (A[0], A[0])):
            assert gb.gdn_group_norm_forward(h, x, A[1], A[2], out, A[4], N, S) == gb.GDN_ERR_ARG
            assert "extent" in gb.gdn_last_error(h)
        for x, stats, dout in ((A[0], A[3], A[4]), (None, None, None)):
            assert gb.gdn_group_norm_backward(h, x, A[1], A[2], stats, dout, A[5], A[6], A[7], N, S) == gb.GDN_ERR_ARG
            assert "extent" in gb.gdn_last_error(h)
    finally:
        gb.gdn_free(h)


@pytest.mark.parametrize("dims", [(), (4,), (4, 4), (2, 2, 2, 2)])
def test_rotary_takes_three_axis_sizes(dims):
    with pytest.raises(ValueError, match="axis_dims"):
        gb.rotary(torch.zeros((1, 2, 3, 8)), dims, grid=(1, 1))
