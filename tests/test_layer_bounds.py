"""The tight bounds of group norm, pinned on the CPU: an fp32 evaluation keeps them, nearly right
ones (planted here) do not."""
import pytest
import torch

import layer_bounds as bounds
import layer_oracle as lo

SIZES = {"rows": (30, 1, 256, 2), "resident": (2, 100, 64, 2), "split": (1, 4000, 64, 2)}


def case(form, offset, seed=91):
    N, S, C, G = SIZES[form]
    g = lo.gen(seed)
    x = torch.randn((N, S, C), generator=g) + offset
    w, b = 1 + 0.3 * torch.randn((C,), generator=g), 0.3 * torch.randn((C,), generator=g)
    how = {"rows": dict(steps=bounds.ROWS, joined=False), "resident": dict(steps=bounds.resident(C // G)),
           "split": dict(steps=bounds.split(C // G, 4, 32))}[form]
    if form == "split":
        how["around"] = bounds.around_pivots(x, G, 128, 32)
    return x, w, b, G, how


def evaluate(x, w, b, G, mistake=None):
    """In fp32, with a mistake in the variance."""
    N, S, C = x.shape
    g = x.reshape(N, S, G, C // G)
    mean = g.mean((1, 3), keepdim=True)
    if mistake == "difference of squares":
        var = (g * g).mean((1, 3), keepdim=True) - mean * mean
    else:
        var = (g - mean).square().mean((1, 3), keepdim=True)
    if mistake == "one in 10^4":
        var = var * (1 + 1e-4)
    rstd = torch.rsqrt(var.clamp_min(0) + 1e-5)
    return ((g - mean) * rstd).reshape(N, S, C) * w + b, torch.cat((mean, rstd), -1)[:, 0]


@pytest.mark.parametrize("offset", [0.0, 1.0, 100.0, 1000.0])
@pytest.mark.parametrize("form", SIZES)
def test_right_arithmetic_passes(form, offset):
    x, w, b, G, how = case(form, offset)
    y, st = evaluate(x, w, b, G)
    o, ob, s, sb = bounds.group_norm(x, w, b, G, "none", **how)
    lo.check("out", y, o, ob)
    lo.check("stats", st, s, sb)


@pytest.mark.parametrize("form,mistake,offset", [(f, "one in 10^4", o) for f in SIZES for o in (0.0, 1.0)] +
                         [(f, "difference of squares", 1000.0) for f in SIZES] + [("rows", "difference of squares", 100.0)])
def test_mistakes_are_caught(form, mistake, offset):
    x, w, b, G, how = case(form, offset)
    y, st = evaluate(x, w, b, G, mistake)
    o, ob, s, sb = bounds.group_norm(x, w, b, G, "none", **how)
    with pytest.raises(AssertionError):
        lo.check("out", y, o, ob)
    with pytest.raises(AssertionError):
        lo.check("stats", st, s, sb)


def test_around_pivots():
    x = torch.tensor([0.0, 1, 2, 3, 4, 5]).reshape(1, 6, 1)
    # stretches of 4 rows by 2: rows 0, 2 around 0; 1, 3 around 1; 4 and 5 around themselves
    assert bounds.around_pivots(x, 1, 4, 2).item() == pytest.approx((4 + 4) / 17.5)
