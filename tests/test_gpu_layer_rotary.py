"""Rotary positions on the GPU against the float64 definition, within derived bounds."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


def run_and_check(label, x, dims, got, positions, **how):
    ref, bound = lo.rotary(x.cpu(), dims, positions.cpu(), **how)
    lo.check(label, got, ref, bound)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("B,T,H,d,dims", [
    (1, 1, 1, 8, (2, 2, 4)),
    (2, 7, 3, 64, (16, 24, 24)),
    (1, 5, 5, 128, (44, 42, 42)),      # odd halves
    (3, 33, 2, 40, (2, 0, 10)),        # most of the head passes through
    (1, 2, 1, 512, (170, 170, 172)),
    (2, 3, 40, 128, (128, 0, 0)),
    (1, 4, 2, 96, (0, 0, 6)),
    (1, 130, 1, 16, (0, 0, 0)),        # nothing turns
    (1, 70, 24, 128, (32, 48, 48)),    # halves of eight, of four and of two elements
    (2, 20, 3, 64, (16, 24, 24)),
    (2, 20, 3, 64, (4, 20, 28)),
    (3, 1400, 2, 32, (8, 8, 8)),       # several tokens a block, the last block not full
])
def test_grid(dtype, halves, B, T, H, d, dims):
    x = lo.randn(lo.gen(1), B, T, H, d, dtype=dtype).cuda()
    y = gb.rotary(x, dims, grid=(3, 5), first_token=4, halves=halves)
    run_and_check("grid", x, dims, y, lo.grid_positions(T, 3, 5, 4), halves=halves)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_given_positions(shared, inverse):
    B, T, H, d, dims = 3, 41, 4, 64, (20, 22, 22)
    g = lo.gen(2)
    pos = torch.randint(-2**31, 2**31, (T, 3) if shared else (B, T, 3), generator=g, dtype=torch.int64).to(torch.int32)
    pos.view(-1)[:4] = torch.tensor([2**31 - 1, -2**31, 0, -1], dtype=torch.int32)
    x = lo.randn(g, B, T, H, d).cuda()
    y = gb.rotary(x, dims, theta=1e6, positions=pos.cuda(), inverse=inverse)
    run_and_check("positions", x, dims, y, pos, theta=1e6, inverse=inverse)


@pytest.mark.parametrize("first", [0, 29 * 52 + 51, 10**9, 2**31 * 30 * 52 - 50])
def test_far_in_the_stream(first):
    dims = (44, 42, 42)
    x = lo.randn(lo.gen(3), 1, 50, 1, 128).cuda()
    y = gb.rotary(x, dims, grid=(30, 52), first_token=first)
    run_and_check(f"first_token {first}", x, dims, y, lo.grid_positions(50, 30, 52, first))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("halves,dims", [(False, (16, 24, 24)), (True, (16, 24, 24)), (True, (10, 22, 26)), (True, (32, 16, 16))])
def test_in_place_in_a_packed_projection(dtype, halves, dims):
    """q and k of a packed row turned in place; v, the padding and the gap stay as they were."""
    B, T, H, d = 2, 70, 3, 64
    buf = lo.randn(lo.gen(4), B, T + 2, 3 * H * d + 16, dtype=dtype).cuda()
    before = buf.clone()
    qk = buf[:, :T, :2 * H * d].unflatten(2, (2 * H, d))
    assert gb.rotary(qk, dims, grid=(5, 7), halves=halves, out=qk) is qk
    run_and_check("in place", before[:, :T, :2 * H * d].unflatten(2, (2 * H, d)), dims, qk,
                  lo.grid_positions(T, 5, 7, 0), halves=halves)
    assert torch.equal(buf[:, :, 2 * H * d:], before[:, :, 2 * H * d:])
    assert torch.equal(buf[:, T:], before[:, T:])


def test_strided_in_and_out_leave_the_rest():
    B, T, H, d, dims = 2, 9, 2, 32, (8, 8, 16)
    x = lo.randn(lo.gen(5), B, T + 1, H * d + 8).cuda()[:, 1:, :H * d].unflatten(2, (H, d))
    out = torch.full((B, T + 3, H * d + 24), 7.0, device="cuda")
    view = out[:, :T, :H * d].unflatten(2, (H, d))
    gb.rotary(x, dims, grid=(2, 2), out=view)
    run_and_check("strided", x, dims, view, lo.grid_positions(T, 2, 2, 0))
    assert (out[:, :T, H * d:] == 7).all() and (out[:, T:] == 7).all()


def test_broadcast_batch_is_read_once_for_each():
    dims = (16, 0, 8)
    x = lo.randn(lo.gen(6), 1, 11, 2, 32).cuda().expand(3, 11, 2, 32)
    y = gb.rotary(x, dims, grid=(1, 4))
    run_and_check("broadcast", x, dims, y, lo.grid_positions(11, 1, 4, 0))


def test_empty():
    assert gb.rotary(torch.empty((2, 0, 3, 16), device="cuda"), (4, 4, 4), grid=(1, 1)).shape == (2, 0, 3, 16)


def test_infinities_and_nan_stay_in_their_pair():
    x = lo.randn(lo.gen(7), 1, 3, 2, 32).cuda()
    x[0, 1, 0, 4], x[0, 2, 1, 9] = float("nan"), float("inf")
    y = gb.rotary(x, (12, 8, 8), grid=(1, 2))
    bad = ~torch.isfinite(y)
    assert bad[0, 1, 0, 4:6].all() and bad[0, 2, 1, 8:10].all() and int(bad.sum()) == 4


@pytest.mark.parametrize("halves", [False, True])
def test_inverse_is_the_gradient(halves):
    """<dy, R x> = <R^-1 dy, x>, and turning back gives x: both to fp32 rounding."""
    g = lo.gen(8)
    x, dy = (lo.randn(g, 2, 37, 3, 64).cuda() for _ in range(2))
    how = dict(axis_dims=(16, 22, 20), grid=(4, 6), first_token=1000, halves=halves)
    y, dx = gb.rotary(x, **how), gb.rotary(dy, inverse=True, **how)
    left, right = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    size = dy.double().abs().sum() * 2 * 8 * lo.U * x.abs().max()
    assert abs(left - right).item() <= size.item()
    back = gb.rotary(y, inverse=True, **how)
    assert (back - x).abs().max().item() <= 4 * 8 * lo.U * 2 * x.abs().max().item()


def test_many_rows():
    """More token rows than one launch has blocks for, checked where they wrap."""
    T, dims = (1 << 20) + 77, (2, 2, 4)
    x = lo.randn(lo.gen(9), 1, 64, 1, 8, dtype="bf16").cuda().repeat(1, T // 64 + 1, 1, 1)[:, :T].contiguous()
    y = gb.rotary(x, dims, grid=(30, 52))
    for a in (0, T // 2, (1 << 20) - 5, T - 40):
        b = min(T, a + 40)
        run_and_check(f"rows {a}", x[:, a:b], dims, y[:, a:b], lo.grid_positions(b - a, 30, 52, a))
