"""Float64 CPU definitions of the operators around the recurrence, with error bounds for
fp32 arithmetic in any order of evaluation, and the comparison the tests use.

u = 2^-24 is the relative error of one fp32 rounding.  An output is rounded once more to
its own type, by at most half a step: finfo(t).eps / 2 relative to the value (and half the
smallest normal number's step where the value is below the normal range)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def out_dtype(dtype):
    return torch.float32 if dtype == "fp32" else torch.bfloat16


def check(label, got, ref, bound):
    """|got - ref| <= bound (absolute, elementwise) + half a step of got's type."""
    assert got.shape == ref.shape, f"{label}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    fi = torch.finfo(got.dtype)
    x = got.detach().cpu().double()
    assert torch.isfinite(x).all(), f"{label}: not finite"
    tol = bound + fi.eps / 2 * (ref.abs() + bound) + fi.tiny * fi.eps
    d = (x - ref).abs()
    bad = d > tol
    if bad.any():
        i = torch.argmax((d - tol).flatten()).item()
        at = tuple(int(k) for k in torch.unravel_index(torch.tensor(i), ref.shape))
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} values off, worst at {at}: "
                             f"{x.flatten()[i]:.9g}, expected {ref.flatten()[i]:.9g} +- {tol.flatten()[i]:.3g}")


# ---- rotary -----------------------------------------------------------------------

def grid_positions(T, height, width, first):
    """[T, 3] positions of a raster, by counting."""
    n = torch.arange(first, first + T, dtype=torch.int64)
    return torch.stack((n // (height * width), (n // width) % height, n % width), -1)


def rotary(x, axis_dims, positions, theta=10000.0, halves=False, inverse=False):
    """x [B, T, H, d] any dtype, positions [B, T, 3] or [T, 3].  (result float64, bound).

    The angle is reduced in 64 bits; the fraction of a turn is rounded to fp32 (at most 1/2, so by
    2^-26 turns = 1e-7 rad), sine and cosine are good to some units of the last place (taken as
    4 u), then two products and a sum: under 8 u per unit of |x| + |y| in all."""
    x = x.double()
    y, bound = x.clone(), torch.zeros_like(x)
    pos = positions.double()
    pos = pos if pos.dim() == 3 else pos[None]
    at = 0
    for axis, n in enumerate(axis_dims):
        for i in range(n // 2):
            e0, e1 = (at + i, at + i + n // 2) if halves else (at + 2 * i, at + 2 * i + 1)
            angle = (pos[:, :, axis] * theta ** (-2.0 * i / n))[:, :, None]
            c, s = torch.cos(angle), torch.sin(angle)
            if inverse:
                s = -s
            y[..., e0] = x[..., e0] * c - x[..., e1] * s
            y[..., e1] = x[..., e0] * s + x[..., e1] * c
            # the 64-bit angle itself: some steps of 2^-53 of the turns passed
            far = 8 * 2.0 ** -53 * angle.abs()
            bound[..., e0] = bound[..., e1] = (8 * U + far) * (x[..., e0].abs() + x[..., e1].abs())
        at += n
    return y, bound


# ---- the diagonal recurrence ------------------------------------------------------

def _wide(y, like):
    y = y.double()
    return y if y.dim() == like.dim() else y[..., None].expand_as(like)


def glr_states(v, beta, decay, state_in=None, reverse=False):
    """Every state in walking order [T, B, H, d] with its start [B, H, d], float64, and the bound of
    an fp32 evaluation in any order: the term that token j adds to state t passes one product for
    b v, t - j products by a decay and at most as many sums, more by a handful where partial results
    are joined: (2 (t - j) + 8) u of its size."""
    v = v.double()
    B, T, H, d = v.shape
    a = _wide(decay, v)
    x = v if beta is None else _wide(beta, v) * v
    order = range(T - 1, -1, -1) if reverse else range(T)
    h = torch.zeros((B, H, d), dtype=torch.float64) if state_in is None else state_in.double()
    size, count = h.abs(), torch.zeros_like(h)
    hs, bounds = torch.empty((T, B, H, d), dtype=torch.float64), torch.empty((T, B, H, d), dtype=torch.float64)
    for k, t in enumerate(order):
        count = a[:, t] * (count + size)  # sum of (t - j) |term|
        size = a[:, t] * size + x[:, t].abs()
        h = a[:, t] * h + x[:, t]
        hs[k], bounds[k] = h, U * (2 * count + 8 * size)
    return hs, bounds


def glr(v, beta, decay, state_in=None, reverse=False):
    """(out [B, T, H, d], its bound, final state, its bound)."""
    hs, bounds = glr_states(v, beta, decay, state_in, reverse)
    B, T, H, d = v.shape
    if T == 0:
        st = torch.zeros((B, H, d), dtype=torch.float64) if state_in is None else state_in.double()
        return hs.permute(1, 0, 2, 3), bounds.permute(1, 0, 2, 3), st, torch.zeros_like(st)
    out, ob = (y.permute(1, 0, 2, 3) for y in (hs, bounds))
    if reverse:
        out, ob = out.flip(1), ob.flip(1)
    return out.contiguous(), ob.contiguous(), hs[-1], bounds[-1]


def glr_grad(v, beta, decay, dout, state_in=None, dstate_out=None, reverse=False):
    """{name: (value, bound)} of dv, dbeta, ddecay, dstate_in."""
    B, T, H, d = v.shape
    vd, a = v.double(), None
    a = _wide(decay, vd)
    b = torch.ones_like(vd) if beta is None else _wide(beta, vd)
    hs, hb = glr_states(v, beta, decay, state_in, reverse)
    h0 = torch.zeros((B, H, d), dtype=torch.float64) if state_in is None else state_in.double()
    order = list(range(T - 1, -1, -1) if reverse else range(T))
    g = torch.zeros_like(h0) if dstate_out is None else dstate_out.double()
    size, count = g.abs(), torch.zeros_like(g)
    res = {n: (torch.empty((B, T, H, d), dtype=torch.float64), torch.empty((B, T, H, d), dtype=torch.float64))
           for n in ("dv", "dbeta", "ddecay")}
    for k in range(T - 1, -1, -1):
        t = order[k]
        do = dout[:, t].double()
        g, size = g + do, size + do.abs()
        gb = U * (2 * count + 8 * size)
        before, bb = (h0, torch.zeros_like(h0)) if k == 0 else (hs[k - 1], hb[k - 1])
        for n, f, fb in (("dv", b[:, t], 0.0), ("dbeta", vd[:, t], 0.0), ("ddecay", before, bb)):
            res[n][0][:, t] = g * f
            res[n][1][:, t] = gb * f.abs() + (g.abs() + gb) * fb + 2 * U * (g * f).abs()
        count = a[:, t] * (count + size)
        g, size = a[:, t] * g, a[:, t] * size
    res["dstate_in"] = (g, U * (2 * count + 8 * size))
    if decay.dim() == 3:  # summed over d: d - 1 sums in some order
        for n in ("dbeta", "ddecay"):
            y, e = res[n]
            res[n] = (y.sum(-1), e.sum(-1) + d * U * (y.abs().sum(-1) + e.sum(-1)))
    return res


# ---- group norm -------------------------------------------------------------------

# Steps of fp32 rounding a reduction may put on a term one after another: the tested samples have at
# most 2^17 values a group, summed by at least 256 threads (or lanes) side by side with a tree over
# them, some 2^9 in all; statistics enter an output through a few such sums.
SUMS = 1024


def _groups(y, G):
    N, S, C = y.shape
    return y.reshape(N, S, G, C // G)


def group_norm(x, weight, bias, G, act, eps=1e-5, sums=SUMS):
    """x [N, S, C]: (out, bound, stats, bound)."""
    x = x.double()
    g = _groups(x, G)
    mean = g.mean((1, 3), keepdim=True)
    var = (g - mean).square().mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = ((g - mean) * rstd).reshape(x.shape)
    w = torch.ones(x.shape[2], dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    z = xhat * w + b
    out = z * torch.sigmoid(z) if act == "silu" else z
    # the mean is off by `sums` u times the mean size, 1/std by `sums` u relative; z * sigmoid(z) has a
    # slope under 1.1 and its exponential and quotient are good to 16 u
    dmean = sums * U * g.abs().mean((1, 3), keepdim=True)
    dx = (dmean * rstd + sums * U * ((g - mean) * rstd).abs()).reshape(x.shape)
    bound = 1.1 * (dx * w.abs() + 4 * U * (xhat * w).abs() + 4 * U * b.abs()) + 16 * U * out.abs()
    stats = torch.cat((mean, rstd), -1)[:, 0]
    sb = torch.cat((dmean, sums * U * rstd * (1 + (mean * rstd) ** 2 * sums * U)), -1)[:, 0]
    return out, bound, stats, sb


def group_norm_grad(x, weight, bias, G, act, dout, eps=1e-5, sums=SUMS):
    """{name: (value, bound)} of dx, dweight, dbias."""
    x, dy = x.double(), dout.double()
    N, S, C = x.shape
    g = _groups(x, G)
    mean = g.mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt((g - mean).square().mean((1, 3), keepdim=True) + eps)
    xhat = ((g - mean) * rstd).reshape(x.shape)
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    z = xhat * w + b
    if act == "silu":
        s = torch.sigmoid(z)
        dz = dy * (s + z * s * (1 - s))
    else:
        dz = dy
    # errors of xhat (as in group_norm) and, through the slope of act' (under 0.5 per unit of z), of dz
    exhat = (sums * U * (g.abs().mean((1, 3), keepdim=True) * rstd + ((g - mean) * rstd).abs())).reshape(x.shape)
    edz = 16 * U * dy.abs() + (0.5 * dy.abs() * (exhat * w.abs() + 4 * U * (z.abs() + b.abs())) if act == "silu" else 0.0)
    t, et = _groups(dz * w, G), _groups(edz * w.abs() + 4 * U * (dz * w).abs(), G)
    xh, exh = _groups(xhat, G), _groups(exhat, G)
    m1, m2 = t.mean((1, 3), keepdim=True), (t * xh).mean((1, 3), keepdim=True)
    dims = dict(dim=(1, 3), keepdim=True)
    em1 = et.mean(**dims) + sums * U * t.abs().mean(**dims)
    em2 = (et * xh.abs() + t.abs() * exh).mean(**dims) + sums * U * (t * xh).abs().mean(**dims)
    dx = rstd * (t - m1 - xh * m2)
    edx = rstd * (et + em1 + xh.abs() * em2 + exh * m2.abs()) + sums * U * rstd * (t.abs() + m1.abs() + (xh * m2).abs())
    dw, db = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    edw = (edz * xhat.abs() + dz.abs() * exhat).sum((0, 1)) + sums * U * (dz * xhat).abs().sum((0, 1))
    edb = edz.sum((0, 1)) + sums * U * dz.abs().sum((0, 1))
    return {"dx": (dx.reshape(x.shape), edx.reshape(x.shape)), "dweight": (dw, edw), "dbias": (db, edb)}


# ---- seeded inputs ----------------------------------------------------------------

def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype="fp32"):
    return torch.randn(shape, generator=g).to(DT[dtype])


def glr_inputs(seed, B, T, H, d, gate="head", dtype="bf16", beta=True, state=True, mean=1.0):
    g = gen(seed)
    shape = (B, T, H) if gate == "head" else (B, T, H, d)
    x = {"v": randn(g, B, T, H, d, dtype=dtype), "decay": torch.sigmoid(randn(g, *shape) + mean),
         "beta": torch.sigmoid(randn(g, *shape)) if beta else None,
         "state": randn(g, B, H, d) if state else None}
    x["dout"] = randn(g, B, T, H, d, dtype="fp32" if dtype == "fp32" else "bf16")
    x["dstate"] = randn(g, B, H, d) if state else None
    return x


def cuda(x):
    return {k: (None if v is None else v.cuda()) for k, v in x.items()}


def raster(first, T, height, width):
    """The same raster counted token by token (checks grid_positions)."""
    f, r = divmod(first, height * width)
    y, c = divmod(r, width)
    out = []
    for _ in range(T):
        out.append((f, y, c))
        c += 1
        if c == width:
            c, y = 0, y + 1
        if y == height:
            y, f = 0, f + 1
    return torch.tensor(out, dtype=torch.int64).reshape(T, 3)


def difference(f, x, dx, step):
    """Central difference of the scalar f along dx."""
    return (f(x + step * dx) - f(x - step * dx)) / (2 * step)


assert math.isclose(U, 5.960464477539063e-08)
