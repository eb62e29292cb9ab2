"""The segments of linear attention: the tests' own rules against the library's, compiled from its source for the
host; workspaces that hold every shorter call; and planted mistakes at a segment's edge that the bounds must notice."""
import os
import random
import re
import subprocess

import pytest
import torch

import linear_cuts as lc
import linear_oracle as no
from gated_deltanet_recurrence_gdn_amd import build

MAIN = r"""
int main() {
    long long B, H, dk, dv, chunks, most, ncu;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &B, &H, &dk, &dv, &chunks, &most, &ncu) == 7) {
        const int f = forward_seg_chunks(B * H, chunks, ncu);
        const GradCut g = grad_cut(B, H, dk, dv, chunks, ncu);
        const bool holds = g.bytes <= grad_most(B, H, dk, dv, most, ncu) && (chunks + f - 1) / f <= forward_most(B * H, most, ncu);
        std::printf("%d %d %d %d %d\n", f, g.seg_chunks, g.nseg, g.group, (int)holds);
    }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    """The source's rules as a program: lines of (B, H, d_k, d_v, chunks, most chunks, CUs) to (chunks of a forward segment, of a
    gradient's, its segments, its group of pairs, whether the workspace for `most` holds them)."""
    with open(os.path.join(build.CSRC, "gdn_linear.hip")) as f:
        src = f.read()
    consts = re.search(r"^constexpr int MAX_SEG_CHUNKS = .*$", src, re.M)[0]
    body = src[src.index("int forward_seg_chunks("):src.index("// The operands of a walk")]
    assert "grad_most" in body
    d = tmp_path_factory.mktemp("cuts")
    (d / "cuts.cpp").write_text("#include <algorithm>\n#include <cstddef>\n#include <cstdio>\nconstexpr int LIN_CHUNK = 64;\n" + consts + "\n" + body + MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-o", str(d / "cuts"), str(d / "cuts.cpp")], check=True)

    def ask(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([str(d / "cuts")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


def test_rules_agree_and_workspaces_hold(rules):
    rng = random.Random(1)
    size = lambda m: min(m, int(m ** rng.random()) + rng.randint(0, 2))  # noqa: E731
    cases = []
    for _ in range(20000):
        most = max(1, size(1 << 24))
        B, H = max(1, size(1 << 8)), max(1, size(1 << 9))
        cases.append((B, H, rng.choice((16, 32, 64, 128)), rng.choice((16, 32, 64, 128)), rng.randint(1, most) if rng.random() < 0.7 else
                      max(1, most - rng.randint(0, 20)), most, rng.choice((256, 256, 304, 64))))
    for case, (f, g, n, group, holds) in zip(cases, rules(cases)):
        B, H, _, _, chunks, _, ncu = case
        assert holds, case
        assert f == lc.forward_cut(B * H, chunks, ncu)[0] and (g, n) == lc.grad_cut(B * H, chunks, ncu), case
        assert g <= lc.MAX_SEG_CHUNKS and 1 <= group <= B * H


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_bounds_notice_a_segment_that_starts_anew(dtype, decay):
    """As GPU tests of segments use the bounds: a state, or its gradient, that does not pass one segment's edge (tokens
    127 and 128, two chunks each)."""
    T, edge = 425, 128
    x = no.linear_inputs(1, 1, T, 2, 16, 16, dtype, mean=5.0)
    if decay == "head":
        x["decay"] = x["decay"][:, 0, 0, None].expand(1, T)[..., None].expand(1, T, 2).contiguous()
    cut = dict(x, decay=x["decay"].clone())
    cut["decay"][:, edge] = 0.0
    right, wrong = no.linear(x, dtype=dtype), no.linear(cut, dtype=dtype)
    for n in ("out", "dq", "dk", "dv", "dlog"):
        t = torch.float32 if dtype == "fp32" or n == "dlog" else torch.bfloat16
        no.check(n, right[n][0].to(t), *right[n])
        with pytest.raises(AssertionError):
            no.check(n, wrong[n][0].to(t), *right[n])
