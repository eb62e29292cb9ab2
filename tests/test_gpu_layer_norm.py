"""Group norm with an activation and its gradient on the GPU against the float64 definition,
within derived bounds."""
import pytest
import torch

import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


def inputs(seed, N, S, C, dtype="bf16", affine=True, offset=0.5):
    g = lo.gen(seed)
    x = (torch.randn((N, S, C), generator=g) * (0.5 + torch.rand((C,), generator=g)) +
         offset * torch.randn((C,), generator=g)).to(lo.DT[dtype])
    w, b = (1 + 0.3 * torch.randn((C,), generator=g), 0.3 * torch.randn((C,), generator=g)) if affine else (None, None)
    return {"x": x, "w": w, "b": b, "dout": lo.randn(g, N, S, C, dtype="fp32" if dtype == "fp32" else "bf16")}


def parity(label, x, G, act="silu", dtype="bf16", eps=1e-5):
    c = lo.cuda(x)
    N, S, C = x["x"].shape
    with gb.GroupNorm(C, G, dtype, act=act, eps=eps, max_N=N) as n:
        out, stats = n.forward(c["x"], c["w"], c["b"])
        bare, none = n.forward(c["x"], c["w"], c["b"], return_stats=False)
        got = n.backward(c["x"], c["w"], c["b"], stats, c["dout"])
        torch.cuda.synchronize()
    assert none is None and torch.equal(out, bare)
    o, ob, st, sb = lo.group_norm(x["x"], x["w"], x["b"], G, act, eps)
    lo.check(f"{label} out", out, o, ob)
    lo.check(f"{label} stats", stats, st, sb)
    ref = lo.group_norm_grad(x["x"], x["w"], x["b"], G, act, x["dout"], eps)
    for name, y, p in zip(("dx", "dweight", "dbias"), got, (True, x["w"], x["b"])):
        if p is None:
            assert y is None
        else:
            lo.check(f"{label} {name}", y, *ref[name])


@pytest.mark.parametrize("N,S,C,G", [
    (1, 1, 8, 1), (1, 1, 8, 8), (5, 1, 64, 4), (131, 1, 256, 2), (3, 1, 4096, 32), (70, 1, 320, 32), (9, 1, 8192, 4),
    (1, 2, 16, 2), (2, 77, 320, 32), (3, 9, 40, 5), (1, 1000, 8, 2), (2, 513, 64, 1), (1, 5000, 128, 32), (2, 1563, 24, 3),
    (40, 64, 512, 8), (1, 300, 8192, 16), (1, 40, 2560, 20), (7, 3, 1000, 125),
    (2, 2, 8192, 8192), (1, 70, 8192, 8192), (2, 6, 4800, 3), (1100, 1, 24, 1), (1, 300, 8, 8), (1030, 17, 1024, 64),
    (77, 1, 80, 1), (300, 1, 24, 1), (41, 1, 1920, 12), (9, 1, 4096, 8), (130, 1, 96, 4), (20, 1, 4480, 7), (30, 700, 64, 16),
])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_shapes(N, S, C, G, act):
    parity("shapes", inputs(31, N, S, C), G, act)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("N,S,C,G", [(33, 1, 128, 8), (2, 50, 64, 4), (1, 3000, 160, 32), (300, 4, 32, 2)])
def test_types(dtype, affine, N, S, C, G):
    parity("types", inputs(32, N, S, C, dtype, affine), G, dtype=dtype)


@pytest.mark.parametrize("N,S,C,G", [(30, 1, 256, 2), (2, 100, 64, 2), (1, 4000, 64, 2)])
def test_means_far_from_zero(N, S, C, G):
    """Means a thousand times the spread: squares are taken around the mean, not subtracted."""
    x = inputs(33, N, S, C, "fp32", offset=0.0)
    x["x"] += 1000.0
    parity("far means", x, G, dtype="fp32")


@pytest.mark.parametrize("N,S,C,G", [(30, 1, 256, 2), (2, 100, 64, 2), (1, 4000, 64, 2)])
def test_one_large_value(N, S, C, G):
    x = inputs(34, N, S, C, "fp32")
    x["x"][:, 0, 0] = 3e4
    parity("outlier", x, G, dtype="fp32")


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("N,S,C,G", [
    (3, 77, 320, 32), (1, 102, 320, 32), (3, 816, 320, 32), (3, 817, 320, 32),  # 8 pieces of 4 groups of 10
    (1, 5, 240, 80), (2, 40, 240, 80), (3, 600, 1280, 32), (2, 77, 4096, 32), (1, 900, 8192, 512), (1, 260, 8192, 8),
    (85, 30, 96, 3), (86, 30, 96, 3), (128, 20, 512, 32), (129, 20, 512, 32), (256, 9, 64, 4), (1, 2, 64, 64),
])
def test_pieces_of_few_samples(dtype, N, S, C, G):
    parity("pieces", inputs(49, N, S, C, dtype), G, dtype=dtype)


@pytest.mark.parametrize("value", [0.0, 10.0, -2.0 ** -20])
def test_constant_groups(value):
    x = inputs(35, 2, 600, 32, "fp32")
    x["x"][..., 8:16] = value
    parity("constant", x, 4, dtype="fp32")


def test_large_activations_do_not_overflow():
    x = inputs(36, 2, 9, 64, "fp32")
    x["w"] *= 300.0
    parity("large z", x, 4, dtype="fp32")


@pytest.mark.parametrize("N,S", [(0, 5), (3, 0), (0, 0)])
def test_empty(N, S):
    with gb.GroupNorm(16, 2, max_N=3) as n:
        x = torch.empty((N, S, 16), dtype=torch.bfloat16, device="cuda")
        w = torch.ones((16,), device="cuda")
        out, stats = n.forward(x, w, w)
        dx, dw, db = n.backward(x, w, w, stats, x)
    assert out.shape == x.shape and dx.shape == x.shape
    assert torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_weight_without_bias_and_gradients_not_wanted():
    x = lo.cuda(inputs(37, 2, 90, 64))
    with gb.GroupNorm(64, 4, max_N=2) as n:
        out, stats = n.forward(x["x"], x["w"], x["b"])
        dx, dw, db = n.backward(x["x"], x["w"], x["b"], stats, x["dout"])
        zero = torch.zeros_like(x["b"])
        assert torch.equal(n.forward(x["x"], x["w"], None)[0], n.forward(x["x"], x["w"], zero)[0])
        assert torch.equal(n.forward(x["x"], None, x["b"])[0], n.forward(x["x"], zero + 1, x["b"])[0])
        for k in range(3):
            bufs = [torch.full_like(y, 5) for y in (dx, dw, db)]
            ptr = [None if i == k else y for i, y in enumerate(bufs)]
            assert gb.gdn_group_norm_backward(n.h, x["x"], x["w"], x["b"], stats, x["dout"], *ptr, 2, 90,
                                              gb.current_stream()) == gb.GDN_OK
            for i, (y, want) in enumerate(zip(bufs, (dx, dw, db))):
                assert (y == 5).all() if i == k else torch.equal(y, want)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("S", [1, 45, 4001])
def test_nan_and_infinity_stay_in_their_group(S, value):
    x = lo.cuda(inputs(38, 4, S, 64))
    x["x"][2, S // 2, 20] = value
    with gb.GroupNorm(64, 4, max_N=4) as n:
        out, stats = n.forward(x["x"], x["w"], x["b"])
        dx, dw, db = n.backward(x["x"], x["w"], x["b"], stats, x["dout"])
    for y in (out, dx):
        bad = torch.isnan(y)
        assert bad[2, :, 16:32].all() and int(bad.sum()) == S * 16
    for y in (dw, db):
        assert torch.isnan(y[16:32]).all() and torch.isfinite(y[:16]).all() and torch.isfinite(y[32:]).all()


def test_frames_with_any_dimensions_between():
    g = lo.gen(39)
    x = lo.randn(g, 2, 3, 5, 7, 32, dtype="bf16").cuda()
    with gb.GroupNorm(32, 4, max_N=2) as n:
        a, sa = n.forward(x)
        b, sb = n.forward(x.view(2, 105, 32))
    assert torch.equal(a.view(2, 105, 32), b) and torch.equal(sa, sb)


@pytest.mark.parametrize("N,S,C,G", [(5, 1, 64, 4), (2, 77, 320, 32), (1, 3001, 24, 3)])
def test_guards(N, S, C, G):
    x = lo.cuda(inputs(40, N, S, C))
    sizes = {"out": N * S * C, "stats": N * G * 2, "dx": N * S * C, "dw": C, "db": C}
    buf = {k: torch.full((m + 512,), 3.0, dtype=torch.bfloat16 if k in ("out", "dx") else torch.float32, device="cuda")
           for k, m in sizes.items()}
    p = {k: y[256:] for k, y in buf.items()}
    with gb.GroupNorm(C, G, max_N=N) as n:
        s = gb.current_stream()
        assert gb.gdn_group_norm_forward(n.h, x["x"], x["w"], x["b"], p["out"], p["stats"], N, S, s) == gb.GDN_OK
        assert gb.gdn_group_norm_backward(n.h, x["x"], x["w"], x["b"], p["stats"], x["dout"], p["dx"], p["dw"], p["db"],
                                          N, S, s) == gb.GDN_OK
        torch.cuda.synchronize()
    for k, m in sizes.items():
        assert (buf[k][:256] == 3).all() and (buf[k][256 + m:] == 3).all(), k
