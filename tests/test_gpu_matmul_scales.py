"""Scales of the 8-bit product far apart: a product of two scales below the normal range of fp32, or beyond
it, must not show where the result itself is within it."""
import pytest
import torch

import linear_oracle as no
from gated_deltanet_recurrence_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu

SCALES = (1.0, 1e-30, 1e30, 2.0 ** -107, 3e-8, 0.0, float("nan"), 1e-12, 5e12, 2.0 ** 120)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (40, 136, 1040), (200, 2056, 144), (2817, 4104, 272)])  # each kernel
def test_scales_far_apart(M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(1)
    a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    a[:, K // 2:] = a[:, :K // 2]
    w[::5, K // 2:] = -w[::5, :K // 2]  # sums of zero
    sa = torch.tensor(SCALES)[torch.randint(len(SCALES), (M,), generator=g)] * (1 + torch.rand(M, generator=g))
    sw = torch.tensor(SCALES)[torch.randint(len(SCALES), (N,), generator=g)] * (1 + torch.rand(N, generator=g))
    b = torch.randn(N, generator=g) if bias else None
    d = lambda x: None if x is None else x.cuda()  # noqa: E731
    got = gb.matmul_int8(d(a), d(sa), d(w), d(sw), bias=d(b), dtype=dtype).double().cpu()
    ref, bound = no.product(a, sa, w, sw, b)
    fi = torch.finfo(torch.float32 if dtype == "fp32" else torch.bfloat16)
    # half a step of the output's type, of its smallest one below its normal range, and of fp32's before it
    tol = bound + fi.eps / 2 * (ref.abs() + bound) + fi.smallest_normal * fi.eps + 2.0 ** -149
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    over = ref.abs() > fi.max * (1 - fi.eps)  # rounds to infinity, or may
    assert (torch.isinf(got) == (ref.abs() > fi.max * (1 + fi.eps)))[~over & ~torch.isnan(ref)].all()
    assert (got.sign() == ref.sign())[over].all()
    fine = ~over & ~torch.isnan(ref)
    bad = fine & ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {int(fine.sum())}; {got[bad][:3].tolist()} for {ref[bad][:3].tolist()}"
