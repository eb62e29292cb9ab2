"""The diagonal gated linear recurrence and its gradient on the GPU against the float64
definition, within derived bounds."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

SAVED = gb.GDN_GLR_SAVED_TOKENS


def parity(label, x, reverse=False, dtype="bf16", grads=True):
    """Forward, saved states and gradient of one set of inputs against the definition."""
    B, T, H, d = x["v"].shape
    gate = "head" if x["decay"].dim() == 3 else "channel"
    c = lo.cuda(x)
    with gb.GLR(B, H, d, dtype, max_T=T, gate=gate, reverse=reverse) as g:
        out, st, saved = g.forward_train(c["v"], c["beta"], c["decay"], state_in=c["state"])
        plain, st2 = g.forward(c["v"], c["beta"], c["decay"], state_in=c["state"])
        got = g.backward(c["v"], c["beta"], c["decay"], saved, c["dout"], c["dstate"]) if grads else None
        torch.cuda.synchronize()
    o, ob, s, sb = lo.glr(x["v"], x["beta"], x["decay"], x["state"], reverse)
    lo.check(f"{label} out", out, o, ob)
    lo.check(f"{label} state_out", st, s, sb)
    assert torch.equal(out, plain) and torch.equal(st, st2), f"{label}: saved states change the result"
    if T:
        hs, hb = lo.glr_states(x["v"], x["beta"], x["decay"], x["state"], reverse)
        start = torch.zeros_like(s) if x["state"] is None else x["state"].double()
        at = range(0, T, SAVED)
        want = torch.stack([start if i == 0 else hs[i - 1] for i in at], 1)
        lo.check(f"{label} saved", saved, want, torch.stack([0 * start if i == 0 else hb[i - 1] for i in at], 1))
    if grads:
        ref = lo.glr_grad(x["v"], x["beta"], x["decay"], x["dout"], x["state"], x["dstate"], reverse)
        for name, y in zip(("dv", "dbeta", "ddecay", "dstate_in"), got):
            if name == "dbeta" and x["beta"] is None:
                assert y is None
            else:
                lo.check(f"{label} {name}", y, *ref[name])


@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("B,T,H,d", [(2, 0, 3, 16), (3, 1, 2, 64), (1, 2, 1, 16), (2, 15, 3, 32), (1, 17, 5, 128),
                                     (1, 127, 2, 64), (2, 128, 1, 32), (1, 129, 9, 16), (1, 1000, 3, 64), (2, 643, 1, 128)])
def test_lengths(gate, reverse, B, T, H, d):
    parity("lengths", lo.glr_inputs(11, B, T, H, d, gate), reverse)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("beta,state", [(True, True), (False, True), (True, False), (False, False)])
def test_types_and_optional_inputs(dtype, gate, beta, state):
    parity("types", lo.glr_inputs(12, 2, 300, 3, 64, gate, dtype, beta, state), dtype=dtype)


@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("kind", ["zero", "one", "tiny", "subnormal", "resets", "near_one", "first_zero"])
def test_decays(gate, kind):
    x = lo.glr_inputs(13, 2, 700, 2, 32, gate, "fp32")
    a = x["decay"]
    if kind == "zero":
        a.zero_()
    elif kind == "one":
        a.fill_(1.0)
    elif kind == "tiny":
        a.fill_(1e-30)
    elif kind == "subnormal":
        a.fill_(2.0 ** -140)
    elif kind == "resets":
        a[:, ::37] = 0.0
    elif kind == "near_one":
        a.fill_(1 - 2.0 ** -12)
    else:
        a[:, 0] = 0.0
    parity(kind, x, dtype="fp32")


@pytest.mark.parametrize("gate", ["head", "channel"])
def test_long_and_wide(gate):
    """Long sequences on few channels, and more channels than the device has lanes for a token tile."""
    parity("long", lo.glr_inputs(14, 1, 20011, 1, 16, gate, mean=4.0))
    parity("wide", lo.glr_inputs(15, 9, 140, 37, 128, gate))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("d,H,beta", [(16, 64, True), (128, 8, False), (32, 33, True)])
def test_long_tiles(dtype, d, H, beta):
    """Enough channels and tokens for the long tiles of gates per head, with a ragged end."""
    parity("long tiles", lo.glr_inputs(22, 16, 2345, H, d, "head", dtype, beta), dtype=dtype)


@pytest.mark.parametrize("reverse", [False, True])
def test_split_calls_carry_the_state_in_place(reverse):
    B, T, H, d = 2, 300, 3, 32
    x = lo.glr_inputs(16, B, T, H, d, "channel", "fp32")
    c = lo.cuda(x)
    cuts = [0, 1, 2, 130, 300]
    parts = list(zip(cuts[:-1], cuts[1:]))
    out, state = torch.empty((B, T, H, d), device="cuda"), c["state"].clone()
    with gb.GLR(B, H, d, "fp32", max_T=T, gate="channel", reverse=reverse) as g:
        for a, b in (reversed(parts) if reverse else parts):
            y, st = g.forward(*(c[k][:, a:b].contiguous() for k in ("v", "beta", "decay")), state_in=state,
                              state_out=state)
            assert st is state
            out[:, a:b] = y
    o, ob, s, sb = lo.glr(x["v"], x["beta"], x["decay"], x["state"], reverse)
    lo.check("split out", out, o, ob)
    lo.check("split state", state, s, sb)


def test_gradients_not_wanted_and_in_place_state_gradient():
    B, T, H, d = 1, 200, 2, 64
    x = lo.cuda(lo.glr_inputs(17, B, T, H, d, "head"))
    with gb.GLR(B, H, d, max_T=T) as g:
        _, _, saved = g.forward_train(x["v"], x["beta"], x["decay"], state_in=x["state"])
        dv, dbeta, ddecay, ds = g.backward(x["v"], x["beta"], x["decay"], saved, x["dout"], x["dstate"])
        for k in range(4):
            bufs = [torch.full_like(y, 5) for y in (dv, dbeta, ddecay)] + [x["dstate"].clone()]
            ptr = [None if i == k else y for i, y in enumerate(bufs)]
            dso = x["dstate"] if k == 3 else bufs[3]  # dstate_in over dstate_out
            assert gb.gdn_glr_backward(g.h, x["v"], x["beta"], x["decay"], saved, x["dout"], dso, *ptr, T,
                                       gb.current_stream()) == gb.GDN_OK
            for i, (y, want) in enumerate(zip(bufs, (dv, dbeta, ddecay, ds))):
                if i != k:
                    assert torch.equal(y, want)
                elif i < 3:
                    assert (y == 5).all()


def test_forward_is_linear_in_v_and_gradient_is_its_difference():
    """Through the GPU's own forward pass in fp32: the difference along dv is exact but for rounding
    (the pass is linear in v), along the decay by a central difference."""
    B, T, H, d = 2, 150, 2, 32
    x = lo.cuda(lo.glr_inputs(18, B, T, H, d, "channel", "fp32"))
    way = {k: torch.randn(x[k].shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda")
           for i, k in enumerate(("v", "decay"))}
    with gb.GLR(B, H, d, "fp32", max_T=T, gate="channel") as g:
        def loss(k, y):
            z = {**x, k: y}
            out, st = g.forward(z["v"], z["beta"], z["decay"], state_in=z["state"])
            return ((out.double() * x["dout"]).sum() + (st.double() * x["dstate"]).sum()).item()
        _, _, saved = g.forward_train(x["v"], x["beta"], x["decay"], state_in=x["state"])
        dv, _, ddecay, _ = g.backward(x["v"], x["beta"], x["decay"], saved, x["dout"], x["dstate"])
        n = x["v"].numel()
        for k, grad, step in (("v", dv, 1.0), ("decay", ddecay, 1e-3)):
            got = (grad.double() * way[k]).sum().item()
            want = lo.difference(lambda y: loss(k, y), x[k], way[k], step)
            # rounding of both losses: n terms of size a few, each off by some u, over the step; the
            # third order of a difference in the decay: step^2 times a loss's size
            tol = 64 * lo.U * n / step + (step ** 2 * n * 8 if k == "decay" else 0)
            assert abs(got - want) <= tol, (k, got, want, tol)


def test_nan_stays_in_its_channel_and_behind_its_token():
    B, T, H, d = 1, 300, 2, 64
    x = lo.cuda(lo.glr_inputs(19, B, T, H, d, "channel", "fp32"))
    x["v"][0, 150, 1, 7] = float("nan")
    with gb.GLR(B, H, d, "fp32", max_T=T, gate="channel") as g:
        out, st = g.forward(x["v"], x["beta"], x["decay"], state_in=x["state"])
    bad = torch.isnan(out)
    assert bad[0, 150:, 1, 7].all() and int(bad.sum()) == T - 150
    assert int(torch.isnan(st).sum()) == 1


def test_guards():
    """Nothing outside the outputs is written, at sizes that end inside every tile."""
    B, T, H, d = 2, 131, 3, 16
    x = lo.cuda(lo.glr_inputs(20, B, T, H, d, "head"))
    sizes = {"out": B * T * H * d, "state": B * H * d, "saved": B * -(-T // SAVED) * H * d, "dv": B * T * H * d, "dbeta": B * T * H,
             "ddecay": B * T * H, "ds": B * H * d}
    buf = {k: torch.full((n + 512,), 3.0, dtype=torch.bfloat16 if k in ("out", "dv") else torch.float32, device="cuda")
           for k, n in sizes.items()}
    p = {k: y[256:] for k, y in buf.items()}
    with gb.GLR(B, H, d, max_T=T) as g:
        s = gb.current_stream()
        assert gb.gdn_glr_forward(g.h, x["v"], x["beta"], x["decay"], x["state"], p["state"], p["saved"], p["out"], T,
                                  s) == gb.GDN_OK
        assert gb.gdn_glr_backward(g.h, x["v"], x["beta"], x["decay"], p["saved"], x["dout"], None, p["dv"], p["dbeta"],
                                   p["ddecay"], p["ds"], T, s) == gb.GDN_OK
        torch.cuda.synchronize()
    for k, n in sizes.items():
        assert (buf[k][:256] == 3).all() and (buf[k][256 + n:] == 3).all(), k


def test_refuses_host_memory():
    x = lo.glr_inputs(21, 1, 4, 1, 16, "head")
    with gb.GLR(1, 1, 16, max_T=4) as g:
        with pytest.raises(ValueError):
            g.forward(x["v"], x["beta"], x["decay"])
        c = lo.cuda(x)
        assert gb.gdn_glr_forward(g.h, x["v"].pin_memory(), None, c["decay"], None, None, None, c["dout"], 4,
                                  gb.current_stream()) == gb.GDN_ERR_ARG
