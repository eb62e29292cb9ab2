"""States behind one strong decay among mild ones, of each token its own: a chunk's factor must not hand its
rounding, which is as large as the logarithm it rounds, on to what came in behind the decay."""
import pytest
import torch

import linear_oracle as no
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

T, STRONG, TERM = 192, 20, 41  # tokens of three chunks, from where the walk starts


def inputs(H, d, dtype, seed=0):
    """A strong decay of each head's own, 2^-99 to 2^-1, and one outer product behind it in the same chunk."""
    g = torch.Generator().manual_seed(seed)
    x = no.linear_inputs(seed, 1, T, H, d, d, dtype, state=False)
    a = 1 - 2.0 ** -12 * torch.rand((1, T, H), generator=g)
    strong = 2.0 ** (-1 - 98 * torch.rand((H,), generator=g))
    return x, a, strong


def check(got, outer, decays):
    """got [H, d, d] against one term times the decays it lives through ([tokens, H]), in steps of fp32.

    A term's roundings, in u: its weight 2 (a power of one step) and 1 (its product), three bf16 parts 1
    and their sums 2 each, the scale 1; then a power of one step, 2, that all chunks' factors together
    are off by, and a product for each of the three chunks.  Logarithms are below 0.03: their roundings are
    2^-29.  With the output's own: 17."""
    want = outer * decays.double().prod(0)[:, None, None]
    err = (got.double().cpu() - want).abs() / want.abs().clamp(min=1e-300)
    assert err.max() <= 17 * no.U, f"{err.max() / no.U:.1f} u, head {int(err.amax((1, 2)).argmax())}"


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_one_strong_decay(d, dtype, reverse):
    H = torch.cuda.get_device_properties(0).multi_processor_count + 64  # pairs enough that a call is one segment
    x, a, strong = inputs(H, d, dtype)
    at = (lambda t: T - 1 - t) if reverse else (lambda t: t)
    c = {n: x[n].cuda() for n in ("q", "k", "v", "dout")}
    with gb.LinearAttention(1, H, d, d, dtype, max_T=T, reverse=reverse, train=True) as op:
        b = a.clone()
        b[:, at(STRONG)] = strong
        v = torch.zeros_like(c["v"])
        v[:, at(TERM)] = c["v"][:, at(TERM)]
        _, state = op.forward(c["q"], c["k"], v, b.cuda())
        o = x["v"][0, at(TERM)].double()[:, :, None] * x["k"][0, at(TERM)].double()[:, None]
        check(state[0], o, b[0, :at(TERM)] if reverse else b[0, at(TERM) + 1:])

        at2 = lambda t: at(T - 1 - t)  # noqa: E731  (the gradient walks the other way)
        b = a.clone()
        b[:, at2(STRONG)] = strong
        do = torch.zeros_like(c["dout"])
        do[:, at2(TERM)] = c["dout"][:, at2(TERM)]
        *_, dstate = op.backward(c["q"], c["k"], c["v"], b.cuda(), do)
        o = x["dout"][0, at2(TERM)].double()[:, :, None] * x["q"][0, at2(TERM)].double()[:, None] * d ** -0.5
        # (1 / sqrt(d) is rounded once where it is no power of two: within the scale's step)
        check(dstate[0], o, b[0, at2(TERM):] if reverse else b[0, :at2(TERM) + 1])
