"""The operators around the recurrence on tensors of more than 2^31 elements: a slice at the far end
against the float64 definition."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


def fill(*shape, seed):
    """Normal values by repeating a block of them (a generator's pass over the whole would be slow)."""
    n = 1
    for k in shape:
        n *= k
    block = lo.randn(lo.gen(seed), 1 << 20, dtype="bf16").cuda()
    return block.repeat(-(-n // block.numel()))[:n].view(shape)


def test_rotary():
    B, T, H, d, dims = 2, 17000, 512, 128, (44, 42, 42)
    x = fill(B, T, H, d, seed=71)
    assert x.numel() > 1 << 31
    y = gb.rotary(x, dims, grid=(30, 52), out=x.clone())
    for t in (0, T - 9):
        ref, bound = lo.rotary(x[1:, t:t + 9, -2:].cpu(), dims, lo.grid_positions(9, 30, 52, t))
        lo.check(f"token {t}", y[1:, t:t + 9, -2:], ref, bound)


def test_diagonal_recurrence():
    B, T, H, d = 2, 9001, 1024, 128
    v, dout = fill(B, T, H, d, seed=72), fill(B, T, H, d, seed=73)
    assert v.numel() > 1 << 31
    g = lo.gen(74)
    decay = torch.sigmoid(torch.randn((B, T, H), generator=g) + 1).cuda()
    with gb.GLR(B, H, d, max_T=T) as r:
        out, state, saved = r.forward_train(v, None, decay)
        dv, _, ddecay, _ = r.backward(v, None, decay, saved, dout)
    last = [y[1:, :, -1:].cpu() for y in (v, decay, dout, out, dv, ddecay)]
    o, ob, s, sb = lo.glr(last[0], None, last[1])
    lo.check("out", last[3], o, ob)
    lo.check("state_out", state[1:, -1:], s, sb)
    ref = lo.glr_grad(last[0], None, last[1], last[2])
    lo.check("dv", last[4], *ref["dv"])
    lo.check("ddecay", last[5], *ref["ddecay"])


def test_group_norm():
    N, S, C, G = 1, 530000, 4096, 512
    x, dout = fill(N, S, C, seed=75), fill(N, S, C, seed=76)
    assert x.numel() > 1 << 31
    w, b = torch.full((C,), 1.5, device="cuda"), torch.full((C,), 0.5, device="cuda")
    with gb.GroupNorm(C, G, max_N=N) as n:
        out, stats = n.forward(x, w, b)
        dx, dw, db = n.backward(x, w, b, stats, dout)
    c = slice(C - C // G, C)  # the last group
    args = (x[:, :, c].cpu(), w[c].cpu(), b[c].cpu(), 1, "silu")
    long = dict(sums=2048)  # a thread adds up some 1,036 rows
    o, ob, st, sb = lo.group_norm(*args, **long)
    lo.check("out", out[:, :, c], o, ob)
    lo.check("stats", stats[:, -1:], st, sb)
    ref = lo.group_norm_grad(*args, dout[:, :, c].cpu(), **long)
    for name, y in (("dx", dx[:, :, c]), ("dweight", dw[c]), ("dbias", db[c])):
        lo.check(name, y, *ref[name])
