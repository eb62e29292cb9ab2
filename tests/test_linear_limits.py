"""The largest sizes that the header allows for 8-bit rows and their product, and the next ones: dry-run calls."""
import pytest

from gated_deltanet_recurrence_gdn_amd import binding as gb

A = [(1 << 56) + (i << 48) for i in range(6)]  # far enough apart for the largest extents
OK, ARG, UNSUP = gb.GDN_OK, gb.GDN_ERR_ARG, gb.GDN_ERR_UNSUPPORTED
TILES = 8388608


def product(M=16, N=64, K=64, stride=None, io=gb.GDN_BF16):
    return gb.gdn_matmul_int8(gb.gdn_matmul_config(-1, N, K, io), A[0], A[1], A[2], A[3], A[4], A[5],
                              N if stride is None else stride, M)


@pytest.mark.parametrize("io", [gb.GDN_F32, gb.GDN_BF16])
@pytest.mark.parametrize("over,code", [
    (dict(M=1, N=1 << 24), OK), (dict(M=1, N=(1 << 24) + 8), UNSUP), (dict(stride=1 << 24), OK), (dict(stride=(1 << 24) + 8), ARG),
    (dict(K=65536), OK), (dict(K=65552), UNSUP),
    # (M / 128 + 1) (N / 128 + 1) up to 2^23: 5,592,404.33 x 1.5, 65,536 x 128
    (dict(M=int((TILES / 1.5 - 1) * 128), N=64), OK), (dict(M=int((TILES / 1.5 - 1) * 128) + 1, N=64), UNSUP),
    (dict(M=(65536 - 1) * 128, N=(128 - 1) * 128), OK), (dict(M=(65536 - 1) * 128 + 1, N=(128 - 1) * 128), UNSUP),
    (dict(M=int((TILES / 1.0625 - 1) * 128), N=8), OK), (dict(M=(1 << 30) + 1, N=8), ARG),
])
def test_product(over, code, io):
    assert product(**over, io=io) == code, gb.gdn_last_error(None)


@pytest.mark.parametrize("N,C,code", [(1 << 24, 8192, OK), ((1 << 24) + 1, 8, ARG), (1, 8192, OK), (1, 8200, UNSUP)])
def test_rows(N, C, code):
    assert gb.gdn_quantize_rows(-1, A[0], gb.GDN_F32, A[1], A[2], N, C) == code
