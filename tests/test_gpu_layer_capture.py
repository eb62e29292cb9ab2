"""First calls of the operators around the recurrence made while a graph is captured: the forms that
ask for more LDS than a launch gets unasked, and one of each other kind.  Every replay, with eager
work between, gives the eager bits."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


def captured(call):
    """Capture call() first, then run it eagerly and compare."""
    torch.zeros(1, device="cuda").add_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = [y for y in call() if y is not None]
    eager = [y.clone() for y in call() if y is not None]
    torch.cuda.synchronize()
    for i in range(3):
        for y in outs:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (y, e) in enumerate(zip(outs, eager)):
            assert torch.equal(y, e), f"replay {i}, output {k}"
        torch.randn(1024, device="cuda").sum().item()
    return eager


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("N,S,C,G", [(3, 1, 8192, 8192), (2, 60, 8192, 8192), (300, 2, 8000, 4000), (5, 1, 512, 8), (1, 5001, 64, 4)])
def test_norm(N, S, C, G, dtype):
    g = lo.gen(101)
    x, dout = lo.randn(g, N, S, C, dtype=dtype).cuda(), lo.randn(g, N, S, C, dtype="fp32" if dtype == "fp32" else "bf16").cuda()
    w, b = torch.rand((C,), generator=g).cuda(), torch.rand((C,), generator=g).cuda()
    with gb.GroupNorm(C, G, dtype, max_N=N) as n:
        def call():
            out, stats = n.forward(x, w, b)
            return (out, stats, *n.backward(x, w, b, stats, dout))
        eager = captured(call)
    o, ob, _, _ = lo.group_norm(x.cpu(), w.cpu(), b.cpu(), G, "silu")
    lo.check("out", eager[0], o, ob)


@pytest.mark.parametrize("T", [1, 50, 2000])
@pytest.mark.parametrize("gate", ["head", "channel"])
def test_recurrence(T, gate):
    x = lo.cuda(lo.glr_inputs(102, 2, T, 3, 64, gate))
    with gb.GLR(2, 3, 64, max_T=T, gate=gate) as r:
        def call():
            out, st, saved = r.forward_train(x["v"], x["beta"], x["decay"], state_in=x["state"])
            return (out, st, *r.backward(x["v"], x["beta"], x["decay"], saved, x["dout"], x["dstate"]))
        captured(call)


@pytest.mark.parametrize("halves", [False, True])
def test_rotary(halves):
    x = lo.randn(lo.gen(103), 2, 40, 3, 64, dtype="bf16").cuda()
    gb.rotary(x[:, :1, :, :8].contiguous(), (2, 2, 4), grid=(1, 1))  # a device's first call checks the device
    captured(lambda: (gb.rotary(x, (18, 22, 24), grid=(5, 7), halves=halves),))
