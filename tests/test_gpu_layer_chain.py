"""The operators around the recurrence as they are used together: positions on q and k of a
packed projection, the recurrence, the norm of its outputs; and a training step through the
diagonal recurrence and the norm.  Eagerly, in a captured graph, on another stream."""
import pytest
import torch

import layer_oracle as lo
import oracle
from gated_deltanet_recurrence_gdn_amd import binding as gb
from gated_deltanet_recurrence_gdn_amd import inputs
from gpu_util import host

pytestmark = pytest.mark.gpu

DIMS, GRID = (16, 24, 24), (10, 13)


def layer(x, g, n, qkv, w, b):
    """The layer around the recurrence: qkv [B, T, 3 H d] is turned in place."""
    B, T, _ = qkv.shape
    qk = qkv[:, :, :2 * g.H * g.d_k].unflatten(2, (2 * g.H, g.d_k))
    gb.rotary(qk, DIMS, grid=GRID, out=qk)
    out, _ = g.forward_packed(qkv, x["beta_logit"], x["decay_logit"])
    y, _ = n.forward(out.view(B * T, g.H * g.d_v), w, b, return_stats=False)
    return y.view(B, T, -1)


def layer_inputs(seed, B, T, H, d):
    x = inputs.make_packed_inputs(B, T, H, d, d, "bf16", seed=seed, pad=0)
    g = lo.gen(seed)
    return x, 1 + 0.1 * torch.randn((H * d,), generator=g), 0.1 * torch.randn((H * d,), generator=g)


def test_layer_matches_the_definitions():
    B, T, H, d = 2, 200, 3, 64
    x, w, b = layer_inputs(51, B, T, H, d)
    c = {k: x[k].cuda() for k in ("beta_logit", "decay_logit")}
    qkv = x["qkv"].contiguous().cuda()
    with gb.GDN(B, H, d, d, "bf16", max_T=T) as g, gb.GroupNorm(H * d, H, max_N=B * T) as n:
        y = layer(c, g, n, qkv, w.cuda(), b.cuda())
        torch.cuda.synchronize()
    q = x["qkv"].contiguous()
    turned, bound = lo.rotary(q[:, :, :2 * H * d].unflatten(2, (2 * H, d)), DIMS, lo.grid_positions(T, *GRID, 0))
    lo.check("positions", qkv[:, :, :2 * H * d].unflatten(2, (2 * H, d)), turned, bound)
    # the recurrence and the norm on the rounded rows that the recurrence read
    o, _ = oracle.forward_packed(qkv.cpu(), x["beta_logit"], x["decay_logit"], H, d, d)
    ref = lo.group_norm(torch.from_numpy(o).reshape(B * T, 1, H * d), w, b, H, "silu")[0].reshape(B, T, H * d)
    # the recurrence's bar (1e-2 relative) through a norm that keeps relative errors
    assert oracle.rel_l2(host(y), ref.numpy()) <= 1.5e-2


def train_step(r, n, x, w, b):
    B, T, H, d = x["v"].shape
    out, st, saved = r.forward_train(x["v"], x["beta"], x["decay"], state_in=x["state"])
    rows = out.view(B * T, H * d)
    y, stats = n.forward(rows, w, b)
    dh, dw, db = n.backward(rows, w, b, stats, x["dout"].view(B * T, H * d))
    return (y, dw, db, st) + r.backward(x["v"], x["beta"], x["decay"], saved, dh.view(B, T, H, d), x["dstate"])


def test_training_step_is_the_gradient():
    """The chained gradient against torch's own of the same definition in float64."""
    B, T, H, d = 2, 150, 2, 32
    x = lo.glr_inputs(52, B, T, H, d, "head", "fp32")
    g = lo.gen(52)
    w, b = 1 + 0.1 * torch.randn((H * d,), generator=g), 0.1 * torch.randn((H * d,), generator=g)
    with gb.GLR(B, H, d, "fp32", max_T=T) as r, gb.GroupNorm(H * d, H, "fp32", max_N=B * T) as n:
        y, dw, db, st, dv, dbeta, ddecay, ds = train_step(r, n, lo.cuda(x), w.cuda(), b.cuda())
        torch.cuda.synchronize()
    p = {k: x[k].double().requires_grad_() for k in ("v", "beta", "decay", "state")}
    w64, b64 = w.double().requires_grad_(), b.double().requires_grad_()
    h, rows = p["state"], []
    for t in range(T):
        h = p["decay"][:, t, :, None] * h + p["beta"][:, t, :, None] * p["v"][:, t]
        rows.append(h)
    o = torch.stack(rows, 1)
    mean, var = o.mean(-1, keepdim=True), o.var(-1, correction=0, keepdim=True)
    z = ((o - mean) / torch.sqrt(var + 1e-5)).reshape(B, T, H * d) * w64 + b64
    y64 = z * torch.sigmoid(z)
    ((y64 * x["dout"].double().reshape(B, T, H * d)).sum() + (h * x["dstate"].double()).sum()).backward()
    for name, got, want in (("y", y, y64.reshape(B * T, -1)), ("state", st, h), ("dw", dw, w64.grad), ("db", db, b64.grad),
                            ("dv", dv, p["v"].grad), ("dbeta", dbeta, p["beta"].grad), ("ddecay", ddecay, p["decay"].grad),
                            ("dstate", ds, p["state"].grad)):
        # fp32 throughout: relative 1e-5 of the whole, as the library's fp32 bar
        assert oracle.rel_l2(host(got), want.detach().numpy()) <= 1e-5, name


def test_captured_and_replayed():
    """A layer and a training step captured together; every replay, with eager work between, gives the
    eager bits."""
    B, T, H, d = 1, 300, 2, 64
    xl, w, b = layer_inputs(53, B, T, H, d)
    c = {k: xl[k].cuda() for k in ("beta_logit", "decay_logit")}
    w, b = w.cuda(), b.cuda()
    fresh = xl["qkv"].contiguous().cuda()
    qkv = fresh.clone()
    x = lo.cuda(lo.glr_inputs(54, B, T, H, d, "channel"))
    frames = lo.randn(lo.gen(55), 1, 5000, 64, dtype="bf16").cuda()
    ones = torch.ones((64,), device="cuda")
    g, n = gb.GDN(B, H, d, d, "bf16", max_T=T), gb.GroupNorm(H * d, H, max_N=B * T)
    r, m = gb.GLR(B, H, d, max_T=T, gate="channel"), gb.GroupNorm(64, 8, max_N=1)

    def step():
        fo, fs = m.forward(frames, ones, ones)
        return (layer(c, g, n, qkv, w, b), *train_step(r, n, x, w, b), fo, *m.backward(frames, ones, ones, fs, frames))

    eager = [y.clone() for y in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    qkv.copy_(fresh)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = step()
    for i in range(4):
        qkv.copy_(fresh)
        for y in outs:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (y, e) in enumerate(zip(outs, eager)):
            assert torch.equal(y, e), f"replay {i}, output {k}"
        torch.randn(1024, device="cuda").sum().item()
        if i == 1:  # the program's own eager call on the same handles, between replays
            qkv.copy_(fresh)
            for y, e in zip(step(), eager):
                assert torch.equal(y, e)
            torch.cuda.synchronize()
    for h in (g, n, r, m):
        h.close()


def test_two_graphs_of_one_handle():
    """Two graphs captured from the same handles and replayed in turn share the handles' workspace."""
    B, T, H, d = 1, 1500, 2, 64
    xs = [lo.cuda(lo.glr_inputs(62 + i, B, T, H, d, "head")) for i in range(2)]
    frames = [lo.randn(lo.gen(64 + i), 1, 6000, 64, dtype="bf16").cuda() for i in range(2)]
    w, ones = torch.ones((H * d,), device="cuda"), torch.ones((64,), device="cuda")
    r, n, m = gb.GLR(B, H, d, max_T=T), gb.GroupNorm(H * d, H, max_N=B * T), gb.GroupNorm(64, 8, max_N=1)

    def step(i):
        fo, fs = m.forward(frames[i], ones, ones)
        return (*train_step(r, n, xs[i], w, w), fo, *m.backward(frames[i], ones, ones, fs, frames[i]))

    eager = [[y.clone() for y in step(i)] for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            outs.append(step(i))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        for y in outs[i]:
            y.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        for k, (y, e) in enumerate(zip(outs[i], eager[i])):
            assert torch.equal(y, e), f"graph {i}, output {k}"
    for h in (r, n, m):
        h.close()


def test_two_handles_on_two_streams():
    """Calls on separate handles may run at the same time: the bits of the same calls in turn."""
    B, T, H, d = 1, 4000, 2, 64
    xs = [lo.cuda(lo.glr_inputs(56 + i, B, T, H, d, "head")) for i in range(2)]
    w = torch.ones((H * d,), device="cuda")
    rs, ns = [gb.GLR(B, H, d, max_T=T) for _ in xs], [gb.GroupNorm(H * d, H, max_N=B * T) for _ in xs]
    frames = [lo.randn(lo.gen(58 + i), 1, 3000, 128, dtype="bf16").cuda() for i in range(2)]

    def step(i):
        return (*train_step(rs[i], ns[i], xs[i], w, w), *ns[i].forward(frames[i], w, w))

    want = [[y.clone() for y in step(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for y, e in zip(outs, want[i]):
                assert torch.equal(y, e)
    for h in rs + ns:
        h.close()


def test_repeated_calls_give_the_same_bits():
    x = lo.cuda(lo.glr_inputs(60, 2, 5000, 3, 32, "head"))
    f = lo.randn(lo.gen(61), 2, 9000, 96, dtype="bf16").cuda()
    w = torch.ones((96,), device="cuda")
    with gb.GLR(2, 3, 32, max_T=5000) as r, gb.GroupNorm(96, 6, max_N=10000) as n:
        def step():
            o, s = n.forward(f, w, w)
            return (*train_step(r, n, x, w, w), o, *n.backward(f, w, w, s, f))
        first = step()
        for _ in range(10):
            for y, e in zip(step(), first):
                assert torch.equal(y, e)
