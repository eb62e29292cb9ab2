"""Group norm in fp32 on the GPU within bounds from the depth of its sums (``layer_bounds``): close
enough to tell squares around the mean from nearly right ones, near and far from zero."""
import pytest
import torch

import layer_bounds as bounds
import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb
from test_layer_bounds import SIZES, case

pytestmark = pytest.mark.gpu


def forward(x, w, b, G, act):
    N, S, C = x.shape
    with gb.GroupNorm(C, G, "fp32", act=act, max_N=N) as n:
        return n.forward(x.cuda(), w.cuda(), b.cuda())


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("offset", [0.0, 1.0, 100.0, 1000.0, -1000.0])
@pytest.mark.parametrize("form", SIZES)
def test_means_near_and_far(form, offset, act):
    x, w, b, G, how = case(form, offset)
    y, st = forward(x, w, b, G, act)
    o, ob, s, sb = bounds.group_norm(x, w, b, G, act, **how)
    lo.check("out", y, o, ob)
    lo.check("stats", st, s, sb)


@pytest.mark.parametrize("form", SIZES)
def test_offsets_of_channels_and_an_outlier(form):
    x, w, b, G, how = case(form, 0.0)
    N, S, C = x.shape
    x = x + 3 * torch.randn((C,), generator=lo.gen(92))
    x[0, 0, 0] = 300.0
    if form == "split":
        how["around"] = bounds.around_pivots(x, G, 128, 32)
    y, st = forward(x, w, b, G, "none")
    o, ob, s, sb = bounds.group_norm(x, w, b, G, "none", **how)
    lo.check("out", y, o, ob)
    lo.check("stats", st, s, sb)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("form", SIZES)
def test_gradient(form, offset, act):
    """Three times the steps: the errors of the mean, and of 1/std through those of the parts' means,
    enter xhat beside those of the sums (offsets up to the spread)."""
    x, w, b, G, how = case(form, offset)
    N, S, C = x.shape
    dout = lo.randn(lo.gen(93), N, S, C)
    with gb.GroupNorm(C, G, "fp32", act=act, max_N=N) as n:
        c = [y.cuda() for y in (x, w, b)]
        _, stats = n.forward(*c)
        got = n.backward(*c, stats, dout.cuda())
    sums = 3 * how["steps"] + 34 * float(torch.as_tensor(how.get("around", 0.0)).max())
    ref = lo.group_norm_grad(x, w, b, G, act, dout, sums=sums)
    for name, y in zip(("dx", "dweight", "dbias"), got):
        lo.check(name, y, *ref[name])
