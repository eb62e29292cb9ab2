"""The C ABI of the operators around the recurrence without a GPU: dry-run calls check every
argument and launch nothing.  Pointers are fake, well-separated addresses."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

GiB = 1 << 30
A = [(1 << 40) + i * GiB for i in range(12)]
OK, ARG, UNSUP, ALIGN, ALIAS = (gb.GDN_OK, gb.GDN_ERR_ARG, gb.GDN_ERR_UNSUPPORTED, gb.GDN_ERR_ALIGN,
                                gb.GDN_ERR_ALIAS)


def rotary(B=2, H=3, d=64, io=gb.GDN_BF16, dims=(16, 24, 24), theta=1e4, flags=0, x=A[0], xts=200, xbs=40000,
           out=A[1], ots=192, obs=19200, pos=None, pbs=0, first=0, height=30, width=52, T=100, device=-1):
    cfg = gb.gdn_rotary_config(device, B, H, d, io, (ctypes.c_int * 3)(*dims), theta, flags)
    return gb.gdn_rotary(cfg, x, xts, xbs, out, ots, obs, pos, pbs, first, height, width, T)


@pytest.mark.parametrize("over", [
    {}, dict(T=0), dict(T=0, x=None, out=None), dict(flags=3), dict(dims=(0, 0, 0)), dict(dims=(64, 0, 0)),
    dict(pos=A[2], pbs=0), dict(pos=A[2], pbs=300), dict(pos=A[2] + 4, pbs=301), dict(io=gb.GDN_FP8, xts=208, xbs=40000),
    dict(out=A[0], ots=200, obs=40000), dict(out=A[0], ots=200, obs=40000, io=gb.GDN_F32),  # in place
    dict(B=1, xbs=0, obs=0), dict(xbs=0), dict(first=10**12), dict(pos=A[2], height=0, width=0, first=-5),
    dict(d=512, H=1, dims=(170, 170, 172), xts=512, ots=512, obs=51200), dict(d=8, H=24, dims=(2, 2, 4)),
])
def test_rotary_accepts(over):
    assert rotary(**over) == OK, gb.gdn_last_error(None)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), ARG), (dict(H=0), ARG), (dict(d=60), UNSUP), (dict(d=0), UNSUP), (dict(d=520), UNSUP), (dict(io=3), UNSUP),
    (dict(dims=(15, 24, 24)), ARG), (dict(dims=(-2, 2, 2)), ARG), (dict(dims=(32, 32, 2)), ARG),
    (dict(dims=(2**31 - 2, 2**31 - 2, 2)), ARG), (dict(theta=0.0), ARG), (dict(theta=0.5), ARG), (dict(theta=float("nan")), ARG),
    (dict(theta=float("inf")), ARG), (dict(flags=4), ARG), (dict(T=-1), ARG), (dict(x=None), ARG), (dict(out=None), ARG),
    (dict(xts=184), ARG), (dict(ots=184), ARG), (dict(xts=1 << 25), UNSUP), (dict(xts=193), ALIGN), (dict(obs=19201), ALIGN),
    (dict(xbs=-8), ARG), (dict(obs=19184), ARG), (dict(x=A[0] + 8), ALIGN), (dict(out=A[1] + 2), ALIGN),
    (dict(pos=A[2] + 2), ALIGN), (dict(pos=A[2], pbs=299), ARG), (dict(pos=A[2], pbs=-300), ARG),
    (dict(out=A[0]), ALIAS), (dict(out=A[0], ots=200, obs=40008), ALIAS), (dict(out=A[0] + 400, ots=200, obs=40000), ALIAS),
    (dict(out=A[0], ots=208, xts=208, obs=40000, io=gb.GDN_FP8), ALIAS), (dict(pos=A[1] + 64), ALIAS),
    (dict(height=0), ARG), (dict(width=0), ARG), (dict(first=-1), ARG), (dict(first=1 << 62), ARG),
    (dict(first=(1 << 31) * 30 * 52 - 50), ARG), (dict(device=-2), ARG), (dict(xbs=1 << 62), ARG),
    (dict(T=1 << 40, obs=1 << 50), UNSUP), (dict(B=2**31 - 1, T=100), UNSUP),
])
def test_rotary_refuses(over, code):
    assert rotary(**over) == code
    assert gb.gdn_last_error(None).startswith("gdn_rotary: ")


def test_rotary_null_config():
    assert gb.library().gdn_rotary(None, None, 0, 0, None, 0, 0, None, 0, 0, 1, 1, 0, None) == ARG


def glr(B=2, H=3, d=64, io=gb.GDN_BF16, gate=1, max_T=1000, flags=0, device=-1):
    return gb.gdn_glr_create(device, B, H, d, io, gate, max_T, flags)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), ARG), (dict(H=0), ARG), (dict(B=32768), UNSUP), (dict(d=48), UNSUP), (dict(H=1 << 15), UNSUP),
    (dict(io=7), UNSUP), (dict(gate=2), ARG), (dict(gate=0), ARG), (dict(max_T=-1), ARG), (dict(flags=1), ARG),
    (dict(flags=8), ARG), (dict(max_T=1 << 60), UNSUP), (dict(max_T=64 << 21), UNSUP), (dict(device=-3), ARG),
])
def test_glr_create_refuses(over, code, capfd):
    st, h = glr(**over)
    assert st == code and h is None
    assert "gdn_glr_create failed" in capfd.readouterr().err


@pytest.fixture(params=[1, 64], ids=["head", "channel"])
def dry_glr(request):
    st, h = glr(gate=request.param, flags=gb.GDN_FLAG_REVERSE if request.param == 1 else 0)
    assert st == OK
    yield h, request.param
    gb.gdn_free(h)


G = dict(v=A[0], beta=A[1], decay=A[2], s_in=A[3], s_out=A[4], saved=A[5], out=A[6], T=100)


def gfwd(h, **over):
    a = {**G, **over}
    return gb.gdn_glr_forward(h, a["v"], a["beta"], a["decay"], a["s_in"], a["s_out"], a["saved"], a["out"], a["T"])


GB = dict(v=A[0], beta=A[1], decay=A[2], saved=A[3], dout=A[4], ds_out=A[5], dv=A[6], dbeta=A[7], ddecay=A[8],
          ds_in=A[9], T=100)


def gbwd(h, **over):
    a = {**GB, **over}
    return gb.gdn_glr_backward(h, a["v"], a["beta"], a["decay"], a["saved"], a["dout"], a["ds_out"], a["dv"],
                               a["dbeta"], a["ddecay"], a["ds_in"], a["T"])


def test_glr_accepts(dry_glr):
    h, _ = dry_glr
    for over in ({}, dict(T=1000), dict(T=1), dict(beta=None), dict(s_in=None), dict(s_out=None), dict(saved=None),
                 dict(s_out=G["s_in"]), dict(T=0, v=None, decay=None, out=None, beta=None)):
        assert gfwd(h, **over) == OK, (over, gb.gdn_last_error(h))
    for over in ({}, dict(beta=None, dbeta=None), dict(ds_out=None), dict(dv=None), dict(dbeta=None), dict(ddecay=None),
                 dict(ds_in=None), dict(ds_in=GB["ds_out"]), dict(T=0, v=None, decay=None, saved=None, dout=None)):
        assert gbwd(h, **over) == OK, (over, gb.gdn_last_error(h))


def test_glr_head_gates_need_four_bytes_only(dry_glr):
    h, gate = dry_glr
    assert gfwd(h, beta=G["beta"] + 4, decay=G["decay"] + 12) == (OK if gate == 1 else ALIGN)


@pytest.mark.parametrize("over,code", [
    (dict(T=1001), ARG), (dict(T=-1), ARG), (dict(v=None), ARG), (dict(decay=None), ARG), (dict(out=None), ARG),
    (dict(v=A[0] + 8), ALIGN), (dict(decay=A[2] + 2), ALIGN), (dict(s_in=A[3] + 4), ALIGN), (dict(saved=A[5] + 4), ALIGN),
    (dict(out=A[0]), ALIAS), (dict(s_out=A[3] + 64), ALIAS), (dict(saved=A[6] + 1024), ALIAS), (dict(saved=A[4]), ALIAS),
    (dict(out=A[2]), ALIAS), (dict(s_out=A[1]), ALIAS),
])
def test_glr_forward_refuses(dry_glr, over, code):
    h, _ = dry_glr
    assert gfwd(h, **over) == code
    assert gb.gdn_last_error(h) != ""


@pytest.mark.parametrize("over,code", [
    (dict(T=1001), ARG), (dict(T=-1), ARG), (dict(v=None), ARG), (dict(decay=None), ARG), (dict(saved=None), ARG),
    (dict(dout=None), ARG), (dict(beta=None), ARG), (dict(dv=A[6] + 8), ALIGN), (dict(ddecay=A[8] + 2), ALIGN),
    (dict(dv=A[4]), ALIAS), (dict(dv=A[0]), ALIAS), (dict(ddecay=A[2]), ALIAS), (dict(dbeta=A[8]), ALIAS),
    (dict(ds_in=A[3]), ALIAS), (dict(ds_in=A[5] + 64), ALIAS),
])
def test_glr_backward_refuses(dry_glr, over, code):
    h, _ = dry_glr
    assert gbwd(h, **over) == code
    assert gb.gdn_last_error(h) != ""


def norm(C=64, Gn=4, io=gb.GDN_BF16, act=1, eps=1e-5, max_N=10, device=-1):
    return gb.gdn_group_norm_create(device, C, Gn, io, act, eps, max_N)


@pytest.mark.parametrize("over,code", [
    (dict(C=60), UNSUP), (dict(C=0), UNSUP), (dict(C=8200), UNSUP), (dict(Gn=3), ARG), (dict(Gn=0), ARG), (dict(Gn=128), ARG),
    (dict(io=9), UNSUP), (dict(act=2), UNSUP), (dict(eps=0.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=1e-40), ARG), (dict(eps=-1e-5), ARG), (dict(eps=float("inf")), ARG), (dict(max_N=-1), ARG),
    (dict(max_N=(1 << 24) + 1), ARG), (dict(device=-2), ARG),
])
def test_group_norm_create_refuses(over, code, capfd):
    st, h = norm(**over)
    assert st == code and h is None
    assert "gdn_group_norm_create failed" in capfd.readouterr().err


@pytest.fixture
def dry_norm():
    st, h = norm()
    assert st == OK
    yield h
    gb.gdn_free(h)


def nfwd(h, x=A[0], w=A[1], b=A[2], out=A[3], stats=A[4], N=5, S=7):
    return gb.gdn_group_norm_forward(h, x, w, b, out, stats, N, S)


def nbwd(h, x=A[0], w=A[1], b=A[2], stats=A[3], dout=A[4], dx=A[5], dw=A[6], db=A[7], N=5, S=7):
    return gb.gdn_group_norm_backward(h, x, w, b, stats, dout, dx, dw, db, N, S)


def test_group_norm_accepts(dry_norm):
    for over in ({}, dict(w=None), dict(b=None), dict(stats=None), dict(N=0, x=None, out=None), dict(S=0), dict(S=1 << 30)):
        if over.get("S") == 1 << 30:  # far apart enough for this extent
            over.update(x=1 << 44, out=1 << 45)
        assert nfwd(dry_norm, **over) == OK, (over, gb.gdn_last_error(dry_norm))
    for over in ({}, dict(w=None, dw=None), dict(dx=None), dict(dw=None), dict(db=None),
                 dict(N=0, x=None, stats=None, dout=None)):
        assert nbwd(dry_norm, **over) == OK, (over, gb.gdn_last_error(dry_norm))


@pytest.mark.parametrize("over,code", [
    (dict(N=-1), ARG), (dict(S=-1), ARG), (dict(N=11), ARG), (dict(x=None), ARG), (dict(out=None), ARG),
    (dict(x=A[0] + 8), ALIGN), (dict(w=A[1] + 4), ALIGN), (dict(stats=A[4] + 8), ALIGN), (dict(out=A[0]), ALIAS),
    (dict(stats=A[1]), ALIAS), (dict(out=A[4]), ALIAS), (dict(S=(1 << 30) + 1), UNSUP),
])
def test_group_norm_forward_refuses(dry_norm, over, code):
    assert nfwd(dry_norm, **over) == code
    assert gb.gdn_last_error(dry_norm) != ""


@pytest.mark.parametrize("over,code", [
    (dict(N=-1), ARG), (dict(N=11), ARG), (dict(x=None), ARG), (dict(stats=None), ARG), (dict(dout=None), ARG),
    (dict(dx=A[5] + 8), ALIGN), (dict(dx=A[4]), ALIAS), (dict(dw=A[7]), ALIAS), (dict(db=A[1]), ALIAS),
])
def test_group_norm_backward_refuses(dry_norm, over, code):
    assert nbwd(dry_norm, **over) == code
    assert gb.gdn_last_error(dry_norm) != ""


def test_handles_of_another_operator_are_refused(dry_norm):
    (_, hg), (_, hr) = glr(), gb.gdn_create(-1, 1, 1, 64, 64, gb.GDN_BF16, 100, gb.GDN_FLAG_BIDI)
    a = A
    for h in (dry_norm, hr):
        assert gfwd(h) == ARG and "another operator" in gb.gdn_last_error(h)
        assert gbwd(h) == ARG
    for h in (hg, hr):
        assert nfwd(h) == ARG and "another operator" in gb.gdn_last_error(h)
        assert nbwd(h) == ARG
    for h in (hg, dry_norm):
        assert gb.gdn_forward(h, a[0], a[1], a[2], a[3], a[4], None, None, a[5], 10, 64) == ARG
        assert gb.gdn_forward_bidi(h, a[0], a[1], a[2], a[3], a[4], a[5], 10, 64) == ARG
        assert gb.gdn_forward_packed(h, a[0], 192, 1920, a[3], a[4], None, None, a[5], 10, 64) == ARG
        assert gb.gdn_forward_bidi_packed(h, a[0], 192, 1920, a[3], a[4], a[5], 10, 64) == ARG
        assert "another operator" in gb.gdn_last_error(h)
    gb.gdn_free(hg)
    gb.gdn_free(hr)
    for f, n in ((gfwd, "gdn_glr_forward"), (gbwd, "gdn_glr_backward"), (nfwd, "gdn_group_norm_forward"),
                 (nbwd, "gdn_group_norm_backward")):
        assert f(None) == ARG and n in gb.gdn_last_error(None)


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        gb.rotary(torch.zeros((1, 2, 3, 8)), (2, 2, 2), grid=(1, 1))
    with pytest.raises(ValueError):
        gb.rotary(torch.zeros((1, 2, 3, 8), dtype=torch.float16), (2, 2, 2), grid=(1, 1))
    with gb.GLR(1, 2, 16, "fp32", max_T=4, device=-1) as g, pytest.raises(ValueError):
        g.forward(torch.zeros((1, 4, 2, 16)), None, torch.zeros((1, 4, 2)))
    with gb.GroupNorm(16, 2, "fp32", device=-1) as n, pytest.raises(ValueError):
        n.forward(torch.zeros((1, 16)))
    with pytest.raises(gb.GDNError):
        gb.GroupNorm(16, 3, "fp32", device=-1)
