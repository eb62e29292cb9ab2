"""What is lost where linear attention takes an fp32 operand as several bf16 parts: the chunked sums with every other step in
64 bits.  Such operands are the weighted rows of a state's update, and the state where the decay's gradient reads it."""
from __future__ import annotations

import torch

CHUNK = 64


def parts(x, n):
    """x as the sum of n bf16 values, each the rounded rest."""
    y, rest = torch.zeros_like(x), x.float()
    for _ in range(n):
        p = rest.bfloat16().float()
        y, rest = y + p.double(), rest - p
    return y


def walk(r1, r2, a1, a2, w, head, whole, S, scale, n):
    """One sweep over chunks [B, H, chunk, token, d] with the state S [B, H, d2, d1]: (last state, a1 . S^T a2 of each token)."""
    dots = []
    for c in range(r1.shape[2]):
        dots.append(((a2[:, :, c] @ parts(S, n)) * a1[:, :, c]).sum(-1) * head[:, :, c] * scale[1])
        S = whole[:, :, c, None, None] * S + parts(r2[:, :, c] * w[:, :, c, :, None] * scale[0], n).transpose(-1, -2) @ r1[:, :, c]
    return S, torch.stack(dots, 2)


def linear(x, n):
    """{state, dstate, dlog} of the call x (decay per token, T a multiple of 64, forwards) with operands in n parts."""
    q, k, v, do = (x[m].double().transpose(1, 2).unflatten(2, (-1, CHUNK)) for m in ("q", "k", "v", "dout"))
    lg = torch.log(x["decay"].double()).transpose(1, 2).unflatten(2, (-1, CHUNK))
    G = lg.cumsum(-1)
    end, sc = G[..., -1:], x["q"].shape[-1] ** -0.5
    whole = end[..., 0].exp()
    S, U = x["state"].double(), x["dstate"].double()
    # forwards: rows k, v, read by q and dout; backwards: rows q, dout, read by k and v, a token's own decay behind it
    back = lambda y: y.flip(2)  # noqa: E731
    fin, xs = walk(k, v, q, do, (end - G).exp(), G.exp(), whole, S, (1.0, sc), n)
    dS, ys = walk(back(q), back(do), back(k), back(v), back(G.exp()), back((end - G).exp()), back(whole), U, (sc, 1.0), n)
    ys = back(ys)
    low = torch.ones((CHUNK, CHUNK), dtype=torch.float64).tril(-1)
    D = ((G[..., :, None] - G[..., None, :]) * low).exp() * low
    W = (q @ k.transpose(-1, -2)) * D * (do @ v.transpose(-1, -2)) * sc
    d = W.sum(-1) - W.sum(-2) + xs
    inside = d.flip(-1).cumsum(-1).flip(-1) + ys.cumsum(-1) - ys
    # the product of state and gradient at a chunk's end, from that at the last one's
    tx, ty = xs.sum(-1), ys.sum(-1)
    later = (tx - ty).flip(-1).cumsum(-1).flip(-1) - (tx - ty)
    base = (fin * U).sum((-1, -2))[..., None] + later - ty
    dlog = (inside + base[..., None]).flatten(2, 3).transpose(1, 2)
    return dict(state=fin, dstate=dS, dlog=dlog)
