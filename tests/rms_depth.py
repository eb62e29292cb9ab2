"""dweight of the root-mean-square norm's gradient with a bound from the depth of the library's sums: a wave (C up to 1,024)
or a block of four walks rows, four waves of a block are added up, and 32 threads a column add the blocks' rows and
then each other's."""
from __future__ import annotations

import linear_oracle as no


def blocks(C, N, ncu):
    rows = N if C > 1024 else -(-N // 4)
    return max(1, min(rows, (2 if C >= 4096 else 4) * ncu))


def depth(C, N, ncu):
    n = blocks(C, N, ncu)
    walked = -(-N // (n if C > 1024 else 4 * n))
    return walked + (0 if C > 1024 else 4) + -(-n // 32) + 5


def dweight(h, dout, ncu, eps=1e-5):
    """(value, bound): a term dout * (h * rstd) is two products and rstd, which is off by what no.rms says."""
    _, _, rstd, rb = no.rms(h, None, eps)
    terms = dout.double() * (h.double() * rstd[:, None])
    N, C = h.shape
    rel = (rb / rstd).max() + (2 + depth(C, N, ncu)) * no.U
    return terms.sum(0), terms.abs().sum(0) * rel
