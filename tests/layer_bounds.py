"""Error bounds of group norm from the depth of its sums, for tests that have to tell a right
fp32 evaluation from a nearly right one (``layer_oracle`` allows 1,024 rounding steps to any)."""
from __future__ import annotations

import torch

from layer_oracle import U, _groups


def unit(D):
    """Channels of a group that a thread joins before LDS: the largest of 8, 4, 2, 1 that divides D."""
    return next(u for u in (8, 4, 2, 1) if D % u == 0)


# Roundings that a term of a group's mean passes, one after another, at most.

ROWS = 8 + 6 + 4  # eight channels of a thread, up to 64 lanes, product and constant


def resident(D):
    """Four rows of a thread, its channels, the threads' units by 64 lanes (1,024 threads: up to 8,192 /
    unit items), a tree over them, some for quotients."""
    return 4 + 8 + -(-8192 // unit(D) // 64) + 6 + 6


def split(D, n, count):
    """n rows of a thread (32 in one sum, four roundings to join each further 32), its channels, 256
    threads' units by 64 lanes and a tree, `count` stretches by 64 lanes and a tree, quotients."""
    return 32 + 4 * -(-n // 32) + 8 + -(-2048 // unit(D) // 64) + 6 + -(-count // 64) + 8 + 8


def around_pivots(x, G, length, R):
    """Sum of squares of what the split form sums up (32 rows of a thread's every R-th around the first of
    them, in stretches of `length`) in units of the squares around the mean: [N, 1, G, 1]."""
    x = x.double()
    i = torch.arange(x.shape[1], device=x.device)
    k = i % length // R
    d = _groups(x - x[:, i - k % 32 * R], G)
    g = _groups(x, G)
    return d.square().sum((1, 3), keepdim=True) / (g - g.mean((1, 3), keepdim=True)).square().sum((1, 3), keepdim=True)


def group_norm(x, weight, bias, G, act, steps, eps=1e-5, joined=True, around=0.0):
    """x [N, S, C] and weight, bias [C] on any device: (out, bound, stats, bound), float64.

    The mean is off by dm = steps u rms(x) at most (rms for the means of parts, of which the joins take
    the squares around: by Cauchy their errors enter the variance by up to 2 dm std; not joined, the
    values' squares around one mean, only by dm^2).  The squares are off by steps u relative, and 34 u
    of what is summed `around` pivots (a sum of 32, a square and a difference).  1/std is off by half of
    the variance's error, 2 u for the reciprocal square root, u for eps and a sum."""
    x = x.double()
    g = _groups(x, G)
    dims = dict(dim=(1, 3), keepdim=True)
    mean = g.mean(**dims)
    var = (g - mean).square().mean(**dims)
    rstd = 1 / torch.sqrt(var + eps)
    dm = steps * U * g.square().mean(**dims).sqrt()
    dvar = (steps + 34 * around) * U * var + dm.square() + (2 * dm * var.sqrt() if joined else 0.0)
    drel = 0.5 * 1.01 * dvar * rstd.square() + 4 * U
    xhat = (g - mean) * rstd
    exhat = 1.01 * (dm * rstd + xhat.abs() * (drel + 2 * U)).reshape(x.shape)
    xhat = xhat.reshape(x.shape)
    z = xhat * weight.double() + bias.double()
    out = z * torch.sigmoid(z) if act == "silu" else z
    ez = exhat * weight.double().abs() + 3 * U * ((xhat * weight.double()).abs() + bias.double().abs())
    bound = 1.1 * ez + 16 * U * out.abs() if act == "silu" else ez
    stats = torch.cat((mean, rstd), -1)[:, 0]
    return out, bound, stats, torch.cat((dm, rstd * drel), -1)[:, 0]
