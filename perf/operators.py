"""The operators around the recurrence, with the cases they are timed on: rotary positions
over time, height and width; the diagonal gated linear recurrence and its gradient; group
norm with an activation, channels last, and its gradient.

``run`` makes one pass: in plain torch operations, or with ``own`` through the library.
"""
import math

import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def _out_dtype(case):
    """fp32 outputs for fp32 inputs, bf16 for bf16 and FP8 inputs."""
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _out_bytes(case):
    return 4 if case["dtype"] == "fp32" else 2


def _in_bytes(case):
    return {"fp32": 4, "bf16": 2, "fp8": 1}[case["dtype"]]


# ---- cases ------------------------------------------------------------------------

def _rotary(B, T, H, d, dims, dtype, given=False, halves=False, inverse=False, pad=0, height=30, width=52,
            first=0, theta=10000.0):
    return dict(op="rotary", B=B, T=T, H=H, d=d, dt=dims[0], dy=dims[1], dx=dims[2], dtype=dtype, given=given,
                halves=halves, inverse=inverse, pad=pad, height=height, width=width, first=first, theta=theta)


def _glr(B, T, H, d, gate, dtype, beta=True, train=False, reverse=False, state=True):
    return dict(op="glr", B=B, T=T, H=H, d=d, gate=gate, dtype=dtype, beta=beta, train=train, reverse=reverse,
                state=state)


def _norm(N, S, C, G, dtype, act="silu", train=False, affine=True):
    return dict(op="norm", N=N, S=S, C=C, G=G, dtype=dtype, act=act, train=train, affine=affine)


def listed():
    cases = [
        # one new token for eight streams, q and k of 20 heads, each stream at its own place
        ("rotary_token", _rotary(8, 1, 40, 128, (44, 42, 42), "bf16", given=True)),
        # one 30 x 52 frame of a streaming call far into the clip, FP8 q and k
        ("rotary_frame_fp8", _rotary(1, 1560, 40, 128, (44, 42, 42), "fp8", first=1560 * 4000)),
        # q and k of 32 heads inside the packed projection of a 21-frame guidance pair
        ("rotary_clip", _rotary(2, 32760, 64, 128, (44, 42, 42), "bf16", pad=4096)),
        # the gradient of ragged images given by their positions, pairs half a section apart
        ("rotary_grad", _rotary(2, 4681, 20, 64, (16, 24, 24), "fp32", given=True, halves=True, inverse=True)),
        # one token of 64 streams, the state carried
        ("glr_step", _glr(64, 1, 20, 128, "head", "bf16")),
        # a 21-frame clip with a gate for each channel
        ("glr_clip", _glr(1, 32760, 20, 128, "channel", "bf16", beta=False)),
        # a training step of the guidance pair, gates per head
        ("glr_train_head", _glr(2, 32760, 32, 128, "head", "bf16", train=True)),
        # a training step at an odd length, gates per channel, the backward direction of a two-way layer
        ("glr_train_channel", _glr(3, 1561, 5, 64, "channel", "fp32", train=True, reverse=True)),
        # the recurrence's outputs of the guidance pair, a group for each of 32 heads
        ("norm_heads", _norm(65520, 1, 4096, 32, "bf16")),
        # a clip's latents in a convolutional block, ten channels a group
        ("norm_clip", _norm(1, 32760, 320, 32, "bf16")),
        # a training step over two clips
        ("norm_train", _norm(2, 32760, 512, 32, "bf16", train=True)),
        # a training step over three small odd images
        ("norm_train_small", _norm(3, 77, 320, 32, "fp32", train=True)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# Channel-tokens of a drawn case: below the largest listed one of its kind.
_MOST = {"rotary": 1 << 28, "glr": 1 << 25, "norm": 2 * 32760 * 4096}


def draw(rng):
    op = rng.choice(("rotary", "rotary", "glr", "glr", "glr", "norm", "norm", "norm"))
    if op == "rotary":
        d = rng.choice((32, 64, 96, 128, 256))
        B, H = _log(rng, 1, 16), _log(rng, 1, 80)
        T = min(_log(rng, 1, 65536), max(1, _MOST[op] // (B * H * d)))
        dx = 2 * rng.randint(1, d // 6)
        dy = 2 * rng.randint(0, d // 6)
        dt = 2 * rng.randint(0, (d - dx - dy) // 2)
        inverse = rng.random() < 0.4
        dtype = rng.choice(("fp32", "bf16", "bf16", "bf16" if inverse else "fp8"))
        return _rotary(B, T, H, d, (dt, dy, dx), dtype, given=rng.random() < 0.5, halves=rng.random() < 0.5,
                       inverse=inverse, pad=16 * rng.randint(0, 40), height=rng.randint(1, 68),
                       width=rng.randint(1, 120), first=rng.choice((0, rng.randint(1, 10**8))),
                       theta=rng.choice((100.0, 10000.0, 1000000.0)))
    if op == "glr":
        d = rng.choice((16, 32, 64, 128))
        B, H = _log(rng, 1, 64), _log(rng, 1, 64)
        T = min(_log(rng, 1, 65536), max(1, _MOST[op] // (B * H * d)))
        return _glr(B, T, H, d, rng.choice(("head", "channel")), rng.choice(("fp32", "bf16", "bf16", "fp8")),
                    beta=rng.random() < 0.6, train=rng.random() < 0.6, reverse=rng.random() < 0.4,
                    state=rng.random() < 0.7)
    G = rng.choice((1, 4, 5, 8, 16, 20, 32))
    C = G * rng.choice((2, 4, 6, 8, 10, 12, 16, 20, 32, 64, 128)) * (4 if G % 4 else 2)
    C = C if C % 8 == 0 else 2 * C
    S = 1 if rng.random() < 0.3 else _log(rng, 2, 400000)
    S = min(S, max(1, _MOST[op] // (4 * C)))
    N = min(_log(rng, 1, 65536 if S == 1 else 64), max(1, _MOST[op] // (4 * C * S)))
    return _norm(N, S, C, G, rng.choice(("fp32", "bf16", "bf16", "fp8")), act=rng.choice(("silu", "silu", "none")),
                 train=rng.random() < 0.6, affine=rng.random() < 0.8)


# ---- inputs -----------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    if case["op"] == "rotary":
        return _prepare_rotary(case, g)
    return _prepare_glr(case, g) if case["op"] == "glr" else _prepare_norm(case, g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_rotary(case, g):
    B, T, H, d = case["B"], case["T"], case["H"], case["d"]
    row = _randn(g, B, T, H * d + case["pad"]).to(DT[case["dtype"]])
    s = dict(case=case, x=row[:, :, :H * d].unflatten(2, (H, d)), positions=None,
             out=torch.empty((B, T, H, d), dtype=_out_dtype(case), device="cuda"))
    if case["given"]:
        high = torch.tensor([5000.0, case["height"], case["width"]], device="cuda")
        s["positions"] = (torch.rand((B, T, 3), generator=g, device="cuda") * high).to(torch.int32)
    return s


def _prepare_glr(case, g):
    B, T, H, d = case["B"], case["T"], case["H"], case["d"]
    dt, odt = DT[case["dtype"]], _out_dtype(case)
    gates = (B, T, H) if case["gate"] == "head" else (B, T, H, d)
    # memories from one token to some hundreds, and now and then a reset (a new sequence)
    mean = torch.rand(gates[2:], generator=g, device="cuda") * 8 - 2
    decay = torch.sigmoid(_randn(g, *gates) + mean)
    decay[torch.rand((B, T), generator=g, device="cuda") < 5e-4] = 0.0
    s = dict(case=case, decay=decay, beta=torch.sigmoid(_randn(g, *gates)) if case["beta"] else None,
             v=_randn(g, B, T, H, d).to(dt), state=_randn(g, B, H, d) if case["state"] else None,
             out=torch.empty((B, T, H, d), dtype=odt, device="cuda"),
             state_out=torch.empty((B, H, d), device="cuda"))
    if case["train"]:
        s["dout"] = _randn(g, B, T, H, d).to(odt)
        s["dstate"] = _randn(g, B, H, d) if case["state"] else None
    if own:
        from gated_deltanet_recurrence_gdn_amd.binding import GLR
        s["op"] = GLR(B, H, d, case["dtype"], max_T=T, gate=case["gate"], reverse=case["reverse"])
    return s


def _prepare_norm(case, g):
    N, S, C = case["N"], case["S"], case["C"]
    # channels with offsets and scales of their own, as a convolution leaves them
    x = _randn(g, N, S, C) * (0.5 + torch.rand((C,), generator=g, device="cuda")) + 0.5 * _randn(g, C)
    s = dict(case=case, x=x.to(DT[case["dtype"]]), w=None, b=None,
             out=torch.empty((N, S, C), dtype=_out_dtype(case), device="cuda"))
    if case["affine"]:
        s["w"], s["b"] = 1 + 0.1 * _randn(g, C), 0.1 * _randn(g, C)
    if case["train"]:
        s["dout"] = _randn(g, N, S, C).to(_out_dtype(case))
    if own:
        from gated_deltanet_recurrence_gdn_amd.binding import GroupNorm
        s["op"] = GroupNorm(C, case["G"], case["dtype"], act=case["act"], max_N=N)
    return s


# ---- one pass ---------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "rotary":
        return _run_rotary(state) if own else _plain_rotary(state)
    if op == "glr":
        return _run_glr(state) if own else _plain_glr(state)
    return _run_norm(state) if own else _plain_norm(state)


def _run_rotary(s):
    from gated_deltanet_recurrence_gdn_amd.binding import rotary
    c = s["case"]
    return rotary(s["x"], (c["dt"], c["dy"], c["dx"]), theta=c["theta"], positions=s["positions"],
                  grid=(c["height"], c["width"]), first_token=c["first"], halves=c["halves"], inverse=c["inverse"],
                  out=s["out"])


def _run_glr(s):
    c = s["case"]
    if not c["train"]:
        return s["op"].forward(s["v"], s["beta"], s["decay"], state_in=s["state"], out=s["out"],
                               state_out=s["state_out"])
    out, state, saved = s["op"].forward_train(s["v"], s["beta"], s["decay"], state_in=s["state"], out=s["out"],
                                              state_out=s["state_out"])
    dv, dbeta, ddecay, dstate = s["op"].backward(s["v"], s["beta"], s["decay"], saved, s["dout"],
                                                 dstate_out=s["dstate"])
    return out, state, dv, dbeta, ddecay, dstate


def _run_norm(s):
    out, stats = s["op"].forward(s["x"], s["w"], s["b"], out=s["out"])
    if not s["case"]["train"]:
        return out
    dx, dw, db = s["op"].backward(s["x"], s["w"], s["b"], stats, s["dout"])
    return (out, dx, dw, db) if s["case"]["affine"] else (out, dx)


# ---- plain forms ------------------------------------------------------------------

def _pairs(case):
    """First and second element of every pair, its axis, and its frequency (64 bits: far positions)."""
    first, second, axis, freq, at = [], [], [], [], 0
    for a, n in enumerate((case["dt"], case["dy"], case["dx"])):
        i = torch.arange(n // 2, device="cuda")
        first.append(at + (i if case["halves"] else 2 * i))
        second.append(at + (i + n // 2 if case["halves"] else 2 * i + 1))
        axis.append(torch.full_like(i, a))
        freq.append(torch.exp(i.double() * (-2.0 / max(n, 1) * math.log(case["theta"]))))
        at += n
    return torch.cat(first), torch.cat(second), torch.cat(axis), torch.cat(freq)


def _plain_rotary(s):
    c = s["case"]
    first, second, axis, freq = _pairs(c)
    if s["positions"] is None:
        t = c["first"] + torch.arange(c["T"], device="cuda")
        area = c["height"] * c["width"]
        pos = torch.stack((t // area, t // c["width"] % c["height"], t % c["width"]), -1)[None]
    else:
        pos = s["positions"]
    angle = pos[..., axis].double() * freq
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    sin = -sin if c["inverse"] else sin
    x = s["x"].float()
    y = x.clone()
    x0, x1 = x[..., first], x[..., second]
    y[..., first] = x0 * cos - x1 * sin
    y[..., second] = x0 * sin + x1 * cos
    return y.to(_out_dtype(c))


def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t over axis 1 from zero, by doubling: after each round every token has taken in
    twice as many before it (a recurrence has no closed elementary form that keeps small decays)."""
    n, step = x.shape[1], 1
    while step < n:
        x = torch.cat((x[:, :step], x[:, step:] + a[:, step:] * x[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return x


def _plain_glr(s):
    c = s["case"]
    head, turn = c["gate"] == "head", c["reverse"]

    def wide(y):
        y = y.unsqueeze(-1) if head and y.dim() == 3 else y
        return torch.flip(y, (1,)) if turn else y

    def back(y, dtype):
        return (torch.flip(y, (1,)) if turn else y).to(dtype)

    odt = _out_dtype(c)
    v, a = wide(s["v"].float()), wide(s["decay"])
    x = v if s["beta"] is None else wide(s["beta"]) * v
    h0 = torch.zeros_like(v[:, 0]) if s["state"] is None else s["state"]
    h = _scan(a, torch.cat((x[:, :1] + a[:, :1] * h0[:, None], x[:, 1:]), 1))
    out, state = back(h, odt), h[:, -1].clone()
    if not c["train"]:
        return out, state
    do = wide(s["dout"].float())
    if s["dstate"] is not None:
        do = torch.cat((do[:, :-1], do[:, -1:] + s["dstate"][:, None]), 1)
    # the gradient's own recurrence runs the other way: g_t = do_t + a_{t+1} g_{t+1}
    later = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    g = torch.flip(_scan(torch.flip(later, (1,)), torch.flip(do, (1,))), (1,))
    da = g * torch.cat((h0[:, None], h[:, :-1]), 1)
    dv, db = g, None
    if s["beta"] is not None:
        dv, db = wide(s["beta"]) * g, g * v
        db = back(db.sum(-1) if head else db, torch.float32)
    return out, state, back(dv, odt), db, back(da.sum(-1) if head else da, torch.float32), a[:, 0] * g[:, 0]


def _plain_norm(s):
    c = s["case"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    x = s["x"].float().view(N, S, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    var = (x - mean).square().mean((1, 3), keepdim=True)
    rstd = 1.0 / torch.sqrt(var + 1e-5)
    xhat = ((x - mean) * rstd).view(N, S, C)
    z = xhat if s["w"] is None else xhat * s["w"] + s["b"]
    sig = torch.sigmoid(z)
    out = (z * sig if c["act"] == "silu" else z).to(_out_dtype(c))
    if not c["train"]:
        return out
    dz = s["dout"].float()
    if c["act"] == "silu":
        dz = dz * sig * (1 + z * (1 - sig))
    dxhat = dz if s["w"] is None else dz * s["w"]
    t = dxhat.view(N, S, G, C // G)
    xh = xhat.view(N, S, G, C // G)
    dx = rstd * (t - t.mean((1, 3), keepdim=True) - xh * (t * xh).mean((1, 3), keepdim=True))
    dx = dx.view(N, S, C).to(_out_dtype(c))
    if s["w"] is None:
        return out, dx
    return out, dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1))


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    ib, ob = _in_bytes(case), _out_bytes(case)
    if case["op"] == "rotary":
        n = case["B"] * case["T"] * case["H"] * case["d"]
        pos = 12 * case["B"] * case["T"] if case["given"] else 0
        return {"bytes": n * (ib + ob) + pos, "flops": 3 * n}
    if case["op"] == "glr":
        n = case["B"] * case["T"] * case["H"] * case["d"]
        gates = (2 if case["beta"] else 1) * 4 * (n if case["gate"] == "channel" else n // case["d"])
        states = 4 * case["B"] * case["H"] * case["d"] * (2 if case["state"] else 1)
        forward = n * (ib + ob) + gates + states
        if not case["train"]:
            return {"bytes": forward, "flops": 3 * n}
        # the gradient reads v, dout and the gates again and writes dv and the gates' gradients
        return {"bytes": forward + n * (ib + 2 * ob) + 2 * gates + states, "flops": 11 * n}
    n = case["N"] * case["S"] * case["C"]
    affine = 8 * case["C"] if case["affine"] else 0
    forward = n * (ib + ob) + affine
    if not case["train"]:
        return {"bytes": forward, "flops": 12 * n}
    return {"bytes": forward + n * (ib + 2 * ob) + 2 * affine, "flops": 36 * n}


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "glr": _exact_glr, "norm": _exact_norm}[case["op"]](s)


def _exact_rotary(s):
    c = s["case"]
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    dev = s["x"].device
    if s["positions"] is not None:
        pos = s["positions"].double()
    else:
        t = torch.arange(c["first"], c["first"] + T, device=dev)
        x = torch.remainder(t, c["width"])
        y = torch.remainder(torch.div(t - x, c["width"], rounding_mode="floor"), c["height"])
        f = torch.div(t, c["width"] * c["height"], rounding_mode="floor")
        pos = torch.stack((f, y, x), -1).double().expand(B, T, 3)
    out = torch.empty((B, T, H, d), dtype=torch.float32 if B * T * H * d > 1 << 28 else torch.float64, device=dev)
    sign = -1.0 if c["inverse"] else 1.0
    for b in range(B):  # a batch element at a time, as complex products: (x + iy) e^{i angle}
        xb, at = s["x"][b].double(), 0
        for a, n in enumerate((c["dt"], c["dy"], c["dx"])):
            if n:
                w = c["theta"] ** (-torch.arange(0, n, 2, dtype=torch.float64, device=dev) / n)
                turn = torch.polar(torch.ones((T, 1, n // 2), dtype=torch.float64, device=dev),
                                   sign * pos[b, :, a, None, None] * w)
                sec = xb[..., at:at + n]
                z = torch.complex(sec[..., :n // 2], sec[..., n // 2:]) if c["halves"] else \
                    torch.view_as_complex(sec.reshape(T, H, n // 2, 2))
                z = z * turn
                out[b, :, :, at:at + n] = torch.cat((z.real, z.imag), -1) if c["halves"] else \
                    torch.view_as_real(z).flatten(2)
            at += n
        out[b, :, :, at:] = xb[..., at:]
    return out


def _exact_glr(s):
    c = s["case"]
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    if B * T * H * d > 1 << 28 or T > 66000:
        return None
    order = range(T - 1, -1, -1) if c["reverse"] else range(T)
    gate = (lambda y: y[..., None]) if c["gate"] == "head" else (lambda y: y)
    dev = s["v"].device
    h = torch.zeros((B, H, d), dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double()
    before = torch.empty((T, B, H, d), dtype=torch.float64, device=dev) if c["train"] else None
    out = torch.empty((B, T, H, d), dtype=torch.float64, device=dev)
    for t in order:
        if before is not None:
            before[t] = h
        x = s["v"][:, t].double()
        h = gate(s["decay"][:, t]).double() * h + (x if s["beta"] is None else gate(s["beta"][:, t]).double() * x)
        out[:, t] = h
    if not c["train"]:
        return out, h
    dv = torch.empty_like(out)
    ddecay = torch.empty(s["decay"].shape, dtype=torch.float64, device=dev)
    dbeta = None if s["beta"] is None else torch.empty_like(ddecay)
    g = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()
    for t in reversed(order):
        g = g + s["dout"][:, t].double()
        da = g * before[t]
        ddecay[:, t] = da.sum(-1) if c["gate"] == "head" else da
        if dbeta is None:
            dv[:, t] = g
        else:
            dv[:, t] = gate(s["beta"][:, t]).double() * g
            db = g * s["v"][:, t].double()
            dbeta[:, t] = db.sum(-1) if c["gate"] == "head" else db
        g = gate(s["decay"][:, t]).double() * g
    return out, h, dv, dbeta, ddecay, g


def _exact_norm(s):
    c = s["case"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    big = N * S * C > 1 << 27
    out = torch.empty((N, S, C), dtype=torch.float32 if big else torch.float64, device=s["x"].device)
    dx = torch.empty_like(out) if c["train"] else None
    ones = torch.ones((C,), dtype=torch.float64, device=out.device)
    w = ones if s["w"] is None else s["w"].double()
    b = 0 * ones if s["b"] is None else s["b"].double()
    dw, db = 0 * ones, 0 * ones
    per = max(1, (1 << 26) // (S * C))
    for n in range(0, N, per):  # some samples at a time
        x = s["x"][n:n + per].double()
        k = x.shape[0]
        grp = x.view(k, S, G, C // G)
        var, mean = torch.var_mean(grp, (1, 3), correction=0, keepdim=True)
        xhat = (grp - mean) / torch.sqrt(var + 1e-5)
        z = xhat.reshape(k, S, C) * w + b
        gate = 1 / (1 + torch.exp(-z))
        out[n:n + per] = z * gate if c["act"] == "silu" else z
        if c["train"]:
            dz = s["dout"][n:n + per].double()
            dz = dz * (gate + z * gate * (1 - gate)) if c["act"] == "silu" else dz
            dw += (dz * xhat.reshape(k, S, C)).sum((0, 1))
            db += dz.sum((0, 1))
            u = (dz * w).view(k, S, G, C // G)
            m = S * (C // G)
            along = (u * xhat).sum((1, 3), keepdim=True) / m
            dx[n:n + per] = ((u - u.sum((1, 3), keepdim=True) / m - xhat * along)
                             / torch.sqrt(var + 1e-5)).reshape(k, S, C)
    if not c["train"]:
        return out
    return (out, dx, dw, db) if c["affine"] else (out, dx)
