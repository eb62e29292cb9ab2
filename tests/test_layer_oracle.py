"""The float64 definitions of the operators around the recurrence, pinned on the CPU: closed
forms, and every gradient formula against central differences."""
import math

import pytest
import torch

import layer_oracle as lo


def test_rotary_closed_forms():
    x = torch.tensor([1.0, 0.0, 0.0, 1.0, 2.0, 3.0, 5.0, 7.0]).reshape(1, 1, 1, 8)
    # position 0 on every axis leaves x; what no axis turns passes through
    y, _ = lo.rotary(x, (4, 2, 0), torch.zeros((1, 3)))
    assert torch.equal(y, x.double())
    # theta = 1: every pair turns by p; a quarter turn takes (1, 0) to (0, 1) and (0, 1) to (-1, 0)
    y, _ = lo.rotary(x, (4, 2, 0), torch.tensor([[math.pi / 2, 0.0, 0.0]], dtype=torch.float64), theta=1.0)
    assert torch.allclose(y.flatten(), torch.tensor([0.0, 1, -1, 0, 2, 3, 5, 7], dtype=torch.float64), atol=1e-15)
    # halves: pairs (0, 2) and (1, 3)
    y, _ = lo.rotary(x, (4, 0, 0), torch.tensor([[math.pi / 2, 0.0, 0.0]], dtype=torch.float64), theta=1.0, halves=True)
    assert torch.allclose(y.flatten()[:4], torch.tensor([0.0, -1, 1, 0], dtype=torch.float64), atol=1e-15)
    # the second pair's frequency is theta^(-2/4)
    y, _ = lo.rotary(x, (4, 0, 0), torch.tensor([[3.0, 9, 9]]), theta=16.0)
    assert y.flatten()[2].item() == pytest.approx(-math.sin(3 / 4), abs=1e-15)


@pytest.mark.parametrize("first,T,height,width", [(0, 13, 2, 3), (5, 20, 3, 4), (7, 4, 1, 1), (1000, 9, 30, 52)])
def test_grid_positions(first, T, height, width):
    assert torch.equal(lo.grid_positions(T, height, width, first), lo.raster(first, T, height, width))


def test_glr_closed_forms():
    one = torch.ones((1, 5, 1, 2), dtype=torch.float64)
    out, _, st, _ = lo.glr(one, None, 0.5 * torch.ones((1, 5, 1)))
    want = torch.tensor([1, 1.5, 1.75, 1.875, 1.9375], dtype=torch.float64)
    assert torch.equal(out[0, :, 0, 0], want) and torch.equal(st[0, 0], want[-1:].expand(2))
    out, _, _, _ = lo.glr(one, None, torch.ones((1, 5, 1)), reverse=True)
    assert torch.equal(out[0, :, 0, 1], torch.tensor([5.0, 4, 3, 2, 1], dtype=torch.float64))
    out, _, _, _ = lo.glr(one, 2 * torch.ones((1, 5, 1)), torch.zeros((1, 5, 1)), torch.full((1, 1, 2), 9.0))
    assert torch.equal(out, 2 * one)  # a zero decay forgets the state


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gate", ["head", "channel"])
def test_glr_gradient_is_the_difference(gate, reverse):
    x = lo.glr_inputs(3, 2, 7, 2, 4, gate, "fp32")
    x = {k: v.double() for k, v in x.items()}

    def loss(**over):
        y = {**x, **over}
        out, _, st, _ = lo.glr(y["v"], y["beta"], y["decay"], y["state"], reverse)
        return ((out * x["dout"]).sum() + (st * x["dstate"]).sum()).item()

    grads = lo.glr_grad(x["v"], x["beta"], x["decay"], x["dout"], x["state"], x["dstate"], reverse)
    g = lo.gen(4)
    for name, grad in (("v", "dv"), ("beta", "dbeta"), ("decay", "ddecay"), ("state", "dstate_in")):
        way = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        want = lo.difference(lambda y: loss(**{name: y}), x[name], way, 1e-5)
        assert (grads[grad][0] * way).sum().item() == pytest.approx(want, rel=1e-7, abs=1e-7), name


def test_group_norm_closed_forms():
    x = torch.tensor([[1.0, 3.0, 10.0, 10.0], [3.0, 1.0, 10.0, 10.0]]).reshape(1, 2, 4)
    y, _, st, _ = lo.group_norm(x, None, None, 2, "none", eps=1e-30)
    assert torch.allclose(y[0, :, :2], torch.tensor([[-1.0, 1.0], [1.0, -1.0]], dtype=torch.float64))
    assert torch.equal(y[0, :, 2:], torch.zeros((2, 2), dtype=torch.float64))  # a constant group
    assert torch.equal(st[0, :, 0], torch.tensor([2.0, 10.0], dtype=torch.float64))
    y, _, _, _ = lo.group_norm(x, torch.full((4,), 2.0), torch.ones(4), 2, "silu")
    z = 1 + 2 / math.sqrt(1 + 1e-5)
    assert y[0, 0, 1].item() == pytest.approx(z / (1 + math.exp(-z)), rel=1e-12)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_gradient_is_the_difference(act):
    g = lo.gen(5)
    x, dy = (torch.randn((2, 5, 12), generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn((12,), generator=g, dtype=torch.float64) for _ in range(2))
    p = {"x": x, "w": w, "b": b}

    def loss(**over):
        y = {**p, **over}
        return (lo.group_norm(y["x"], y["w"], y["b"], 3, act)[0] * dy).sum().item()

    grads = lo.group_norm_grad(x, w, b, 3, act, dy)
    for name, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        way = torch.randn(p[name].shape, generator=g, dtype=torch.float64)
        want = lo.difference(lambda y: loss(**{name: y}), p[name], way, 1e-5)
        assert (grads[grad][0] * way).sum().item() == pytest.approx(want, rel=1e-7, abs=1e-7), name


@pytest.mark.parametrize("mistake", ["value", "shape", "nan"])
def test_check_catches(mistake):
    ref = torch.randn((3, 4), generator=lo.gen(6)).double()
    got = ref.to(torch.bfloat16)
    lo.check("rounded", got, ref, torch.zeros_like(ref))
    if mistake == "value":
        got[1, 2] *= 1 + 2.0 ** -6
    elif mistake == "shape":
        got = got[:2]
    else:
        got[0, 0] = float("nan")
    with pytest.raises(AssertionError):
        lo.check(mistake, got, ref, torch.zeros_like(ref))
