"""The forms of the operators around the recurrence that only calls of some size take, at sizes
formed from the device's CU count, with ragged ends: long tiles of the diagonal recurrence,
several rounds of the norm's rows and split forms, many rows of a thread.

Each test states the launch rule that it relies on and asserts that its size takes the form."""
import pytest
import torch

import layer_bounds as bounds
import layer_oracle as lo
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def repeated(g, *shape, dtype="bf16"):
    """Normal values on the GPU: a block of them repeated with a period that no row or tile divides."""
    n = 1
    for k in shape:
        n *= k
    block = lo.randn(g, 999983, dtype=dtype).cuda()
    return block.repeat(-(-n // block.numel()))[:n].view(shape)


# ---- the diagonal recurrence ------------------------------------------------------

# Tokens of a wave with gates per head, and the least tiles of a CU, from which on a call takes
# them (fewer: 16 forward, 8 backward); a tile is eight waves.
FORWARD, BACKWARD, TILES_A_CU = {"fp32": 32, "bf16": 64, "fp8": 64}, 16, 4


@pytest.mark.parametrize("dtype,beta,reverse,H,d",
                         [(t, b, r, 8, 128) for t in ("fp32", "bf16", "fp8") for b in (True, False) for r in (False, True)] +
                         [("bf16", True, False, 66, 16), ("fp8", True, True, 66, 16),  # slabs that end inside
                          ("bf16", False, True, 17, 64), ("fp32", True, False, 17, 64)])
def test_long_tiles(dtype, beta, reverse, H, d):
    slabs = -(-H * d // 128)
    T = 4 * 8 * FORWARD[dtype] + 37
    B = -(-TILES_A_CU * cus() // (5 * slabs))
    for tokens in (FORWARD[dtype], BACKWARD):
        assert T >= 8 * tokens and B * slabs * -(-T // (8 * tokens)) >= TILES_A_CU * cus() and B * slabs > 8
    g = lo.gen(81)
    odt = "fp32" if dtype == "fp32" else "bf16"
    v, dout = repeated(g, B, T, H, d, dtype=dtype), repeated(g, B, T, H, d, dtype=odt)
    decay = torch.sigmoid(torch.randn((B, T, H), generator=g) + 1).cuda()
    bt = torch.sigmoid(torch.randn((B, T, H), generator=g)).cuda() if beta else None
    state, dstate = repeated(g, B, H, d, dtype="fp32"), repeated(g, B, H, d, dtype="fp32")
    with gb.GLR(B, H, d, dtype, max_T=T, reverse=reverse) as r:
        out, st, saved = r.forward_train(v, bt, decay, state_in=state)
        bare, _ = r.forward(v, bt, decay, state_in=state)
        dv, dbeta, ddecay, ds = r.backward(v, bt, decay, saved, dout, dstate)
    assert torch.equal(out, bare)

    def some(y):  # three heads as a batch of their own: heads do not know of each other
        at = (0, 0), (B // 2, H // 2), (B - 1, H - 1)
        head = 2 if y.shape[1] == T else 1
        return torch.cat([y[b:b + 1].narrow(head, h, 1) for b, h in at]).cpu()

    x = [None if y is None else some(y) for y in (v, bt, decay)]
    o, ob, s, sb = lo.glr(*x, some(state), reverse)
    lo.check("out", some(out), o, ob)
    lo.check("state_out", some(st), s, sb)
    ref = lo.glr_grad(*x, some(dout), some(state), some(dstate), reverse)
    for name, y in (("dv", dv), ("dbeta", dbeta), ("ddecay", ddecay), ("dstate_in", ds)):
        if y is not None:
            lo.check(name, some(y), *ref[name])


# ---- group norm -------------------------------------------------------------------

def check(label, got, ref, bound):
    """layer_oracle.check on the device."""
    fi = torch.finfo(got.dtype)
    tol = bound + fi.eps / 2 * (ref.abs() + bound) + fi.tiny * fi.eps
    bad = ~((got.double() - ref).abs() <= tol)
    assert got.shape == ref.shape and not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} values off"


def norm_inputs(seed, N, S, C, dtype, offset=0.5):
    g = lo.gen(seed)
    x = (repeated(g, N, S, C, dtype="fp32") + offset * torch.randn((C,), generator=g).cuda()).to(lo.DT[dtype])
    w, b = ((k + 0.3 * torch.randn((C,), generator=g)).cuda() for k in (1, 0))
    return x, w, b, repeated(g, N, S, C, dtype="fp32" if dtype == "fp32" else "bf16")


def norm_parity(x, w, b, dout, G, act, dtype, steps, sums, part=slice(None), around=(), far=3):
    """Forward and gradient against the float64 definition on the device, on the channels `part` (whole
    groups).  sums: the depth of the gradient's, dweight's and dbias' sums included.  around: the
    (length, R) of the split form's stretches.

    xhat is off by steps u (m + |xhat| (1/2 + r)) for m and r the mean and rms size over the std (the mean;
    1/std through the squares and the means of parts), layer_oracle's gradient by its sums u (m + |xhat|):
    three times the steps cover it where r is some 1, 1 + |xhat| times the steps (`far`) where m = r is large."""
    N, S, C = x.shape
    with gb.GroupNorm(C, G, dtype, act=act, max_N=N) as n:
        out, stats = n.forward(x, w, b)
        bare, _ = n.forward(x, w, b, return_stats=False)
        dx, dw, db = n.backward(x, w, b, stats, dout)
    assert torch.equal(out, bare)
    c = torch.arange(C)[part]
    g0, g1 = int(c[0]) // (C // G), int(c[-1]) // (C // G) + 1
    args = (x[..., part], w[part], b[part], g1 - g0, act)
    around = torch.stack([bounds.around_pivots(x[..., part], g1 - g0, *k) for k in around]).amax(0) if around else 0.0
    o, ob, st, sb = bounds.group_norm(*args, steps, around=around)
    check("out", out[..., part], o, ob)
    check("stats", stats[:, g0:g1], st, sb)
    del o, ob
    extra = 34 * float(torch.as_tensor(around).max())
    ref = lo.group_norm_grad(*args, dout[..., part], sums=far * sums + extra)
    for name, y in (("dx", dx[..., part]), ("dweight", dw[part]), ("dbias", db[part])):
        check(name, y, *ref[name])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("C,G,act", [(4096, 32, "silu"), (480, 20, "none"), (64, 8, "silu")])
def test_rows_form_over_several_rounds(dtype, C, G, act):
    """Blocks of 24 waves a CU forward (16 for the gradient) take four rows a thread (two) in a round:
    two rounds and a ragged third (six and more); 16, 3 of 4 and one lane a group."""
    P = C // G // 8
    L = 1
    while L < P:
        L *= 2
    threads = max(256, -(-G * L // 64) * 64)
    R = threads // (G * L)
    blocks = 16 * cus() * 64 // threads
    N = 2 * 4 * (blocks * 3 // 2) * R + 77
    x, w, b, dout = norm_inputs(82, N, 1, C, dtype)
    # dweight: the rows of a thread, of a block, of 32 threads over the blocks, and a tree
    norm_parity(x, w, b, dout, G, act, dtype, bounds.ROWS, -(-N // (blocks * R)) + R + blocks // 32 + 5 + bounds.ROWS)


@pytest.mark.parametrize("dtype,N,S,C,G", [("bf16", 1030, 1100, 32, 4), ("fp32", 1030, 40, 1024, 64), ("fp8", 1030, 40, 1024, 64),
                                           ("bf16", 2100, 40, 1000, 100)])
def test_split_form_over_rounds_of_samples(dtype, N, S, C, G):
    """The split form takes 1,024 samples at a time and adds dweight and dbias up over such rounds.
    Samples too large for one block (more than four rows of each of 1,024 threads), more of them than
    CUs."""
    V = C // 8
    assert N > 1024 > cus() and S > 4 * (1024 // V)
    x, w, b, dout = norm_inputs(83, N, S, C, dtype)
    R = max(256, -(-V // 64) * 64) // V
    n = -(-S // R)
    # whole samples a stretch in the first rounds; down to four rows a thread in the last, of few samples
    lengths = [rows * 4 * R for rows in range(1, -(-S // (4 * R)) + 1)]
    steps = bounds.split(C // G, n, len(lengths))
    norm_parity(x, w, b, dout, G, "silu", dtype, steps, steps + R + 1024 // 32 + 8, around=[(k, R) for k in lengths])


@pytest.mark.parametrize("dtype,offset,outlier,C,G,n", [
    ("fp32", 0.5, None, 2048, 16, 72), ("fp32", 1000.0, None, 2048, 16, 72), ("fp32", 0.5, 3e4, 2048, 16, 72),
    ("bf16", 0.5, None, 2048, 16, 72), ("fp32", 0.5, None, 96, 16, 36), ("bf16", 3.0, None, 96, 16, 36)])
def test_split_form_of_many_rows_a_thread(dtype, offset, outlier, C, G, n):
    """More than 32 rows of a thread, which it sums up around a pivot each and joins, four in flight; the
    last stretch a single row (C = 2048), and threads without a row in it (C = 96)."""
    V = C // 8
    R = max(256, -(-V // 64) * 64) // V
    stretches = 16 * cus() * 64 // 256  # wanted
    S = (stretches - 24) * n * R + 1
    length = -(-S // (stretches * 4 * R)) * 4 * R  # whole rounds of four rows
    assert length == n * R and n > 32
    x, w, b, dout = norm_inputs(84, 1, S, C, dtype, 0.0 if offset > 100 else offset)
    if offset > 100:
        x += offset
    if outlier:
        x[0, 5, 0] = outlier
    count = -(-S // length)
    steps = bounds.split(C // G, n, count)
    D = C // G
    for part in (slice(0, D), slice(C - D, C)):
        norm_parity(x, w, b, dout, G, "silu", dtype, steps, steps + n + R + count // 32 + 5, part, [(length, R)],
                    far=8 if offset > 100 else 3)  # values up to 5 std


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp8"])
def test_resident_form_of_more_samples_than_blocks(dtype):
    """A launch has at most 2^20 blocks of samples."""
    N, S, C, G = (1 << 20) + 77, 2, 16, 4
    x, w, b, dout = norm_inputs(85, N, S, C, dtype)
    blocks = 16 * cus()  # of the gradient, a wave each
    norm_parity(x, w, b, dout, G, "silu", dtype, bounds.resident(C // G), bounds.resident(C // G) + -(-N // blocks) + blocks // 32 + 64)


@pytest.mark.parametrize("N,C,G", [(70, 8192, 1024), (1300, 4096, 2048), (3, 8192, 8192)])
def test_rows_of_more_groups_than_the_rows_form_takes(N, C, G):
    x, w, b, dout = norm_inputs(86, N, 1, C, "fp32", offset=0.0)
    steps = bounds.resident(C // G)
    norm_parity(x, w, b, dout, G, "none", "fp32", steps, steps + 64 + N)


# ---- the diagonal recurrence over many tiles ---------------------------------------

@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gate", ["head", "channel"])
@pytest.mark.parametrize("H", [1, 11])
def test_long_look_back(H, gate, reverse):
    """79 tiles forward and 157 for the gradient: windows of 16 tiles (11 slabs) and of 64 (one)."""
    B, T, d = 1, 10011, 128
    x = lo.glr_inputs(87, B, T, H, d, gate, mean=4.0)
    c = lo.cuda(x)
    with gb.GLR(B, H, d, max_T=T, gate=gate, reverse=reverse) as r:
        out, st, saved = r.forward_train(c["v"], c["beta"], c["decay"], state_in=c["state"])
        got = r.backward(c["v"], c["beta"], c["decay"], saved, c["dout"], c["dstate"])
    h = slice(H - 1, H)
    y = {k: (z[:, h] if k in ("state", "dstate") else z[:, :, h]) for k, z in x.items()}
    o, ob, s, sb = lo.glr(y["v"], y["beta"], y["decay"], y["state"], reverse)
    lo.check("out", out[:, :, h], o, ob)
    lo.check("state_out", st[:, h], s, sb)
    ref = lo.glr_grad(y["v"], y["beta"], y["decay"], y["dout"], y["state"], y["dstate"], reverse)
    for name, z in zip(("dv", "dbeta", "ddecay", "dstate_in"), got):
        lo.check(name, z[:, h] if name == "dstate_in" else z[:, :, h], *ref[name])
