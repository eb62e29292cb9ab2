"""Linear attention cut into segments of several chunks, the last one shorter: every token of every output of some heads,
forward and gradient, states and their gradients in, both directions, against the float64 definition."""
import pytest
import torch

import linear_cuts as lc
import linear_oracle as no
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

NAMES = ("out", "state", "dq", "dk", "dv", "dlog", "dstate")


def inputs(seed, B, T, H, dk, dv, dtype, decay):
    """On the device; memories of some hundred tokens, so that much passes a segment's edge."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt, odt = no.DT[dtype], no.out_dtype(dtype)
    k = r(B, T, H, dk)
    a = torch.sigmoid(r(H) + 5) if decay == "head" else torch.sigmoid(r(B, T, H) + 5)
    return dict(q=r(B, T, H, dk).to(dt), k=(k / k.norm(dim=-1, keepdim=True)).to(dt), v=r(B, T, H, dv).to(dt), decay=a,
                state=r(B, H, dv, dk), dout=r(B, T, H, dv).to(odt), dstate=r(B, H, dv, dk))


def parity(x, dtype, reverse, heads):
    B, T, H, dk = x["q"].shape
    dv, per_head = x["v"].shape[-1], x["decay"].dim() == 1
    with gb.LinearAttention(B, H, dk, dv, dtype, max_T=T, decay="head" if per_head else "token", reverse=reverse,
                            train=True) as op:
        got = op.forward(x["q"], x["k"], x["v"], x["decay"], state_in=x["state"])
        got += op.backward(x["q"], x["k"], x["v"], x["decay"], x["dout"], state_in=x["state"], dstate_out=x["dstate"])
        torch.cuda.synchronize()
    at = torch.tensor(heads, device="cuda")
    pick = lambda n, y: y[at] if n in ("decay", "dlog") and per_head else y.index_select(1 if "state" in n else 2, at)  # noqa: E731
    ref = no.linear({n: pick(n, y).cpu() for n, y in x.items()}, reverse, dtype)
    for n, y in zip(NAMES, got):
        y = pick(n, y)
        no.check(n, y, *ref[n])
        bar = 5e-3 if y.dtype is torch.bfloat16 else 1e-5
        assert no.rel_l2(y, ref[n][0]) <= bar, f"{n}: rel-L2 {no.rel_l2(y, ref[n][0]):.2e}"


def cuts(pairs, chunks):
    ncu = torch.cuda.get_device_properties(0).multi_processor_count
    return lc.forward_cut(pairs, chunks, ncu), lc.grad_cut(pairs, chunks, ncu)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype,decay", [("bf16", "token"), ("bf16", "head"), ("fp32", "token"), ("fp32", "head"), ("fp8", "token")])
@pytest.mark.parametrize("B,H,T,dk,dv", [
    (2, 20, 425, 16, 16),    # segments of 2, 2, 2 and 1 chunks
    (3, 20, 683, 32, 16),    # 3, 3, 3, 2
    (2, 80, 1050, 16, 64),   # 6, 6, 5
])
def test_ragged_segments(B, H, T, dk, dv, dtype, decay, reverse):
    chunks = lc.up(T, 64)
    for s, n in cuts(B * H, chunks):
        assert s > 1 and n > 2 and chunks % s and T % 64
    parity(inputs(1, B, T, H, dk, dv, dtype, decay), dtype, reverse, [0, H // 2, H - 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ragged_segments_of_wide_heads(dtype):
    """Both head dims of 128: eight waves a block, segments of 3, 3, 3 and 2 chunks."""
    B, H, T = 2, 30, 683
    (f, _), (g, n) = cuts(B * H, lc.up(T, 64))
    assert f == g == 3 and n == 4
    parity(inputs(2, B, T, H, 128, 128, dtype, "token"), dtype, False, [0, H - 1])


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("reverse", [False, True])
def test_groups_of_pairs(decay, reverse):
    """More pairs than the gradient's workspace holds at a time: several groups, several segments each, a last group of
    fewer pairs, and a decay's gradient that sums over them."""
    B, H, T, d = 3, 683, 1050, 128
    chunks = lc.up(T, 64)
    s, n = cuts(B * H, chunks)[1]
    pair_bytes = ((2 * n + 1) * d * d + 6 * chunks * 64 + 4 * n) * 4 + 8 * n
    group = (512 << 20) // pair_bytes
    assert n > 1 and chunks % s and group < B * H and B * H % group
    parity(inputs(3, B, T, H, d, d, "bf16", decay), "bf16", reverse, [0, group % H - 1, H - 1])
