"""The device assembly of the library's sources, compiled as the build does, for tests that look at
what orders its memory operations.  No GPU is needed."""
from __future__ import annotations

import functools
import os
import re
import subprocess

from gated_deltanet_recurrence_gdn_amd import build


@functools.lru_cache(maxsize=None)
def kernels(source: str) -> dict[str, tuple[str, ...]]:
    """{mangled name: lines without comments} of the kernels of csrc/<source>; labels are lines of their own."""
    cmd = [build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", "-"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    res, name, lines = {}, None, []
    for line in r.stdout.splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"(_Z\w+):$", line)
        if m:
            name, lines = m[1], []
        elif name and line.startswith(".Lfunc_end"):
            res[name], name = tuple(lines), None
        elif name and line and (line.startswith(".LBB") or not line.startswith(".")):
            lines.append(line)
    return res


def _registers(operand: str) -> set[str]:
    m = re.match(r"([av])\[(\d+):(\d+)\]$", operand) or re.match(r"([av])(\d+)()$", operand)
    return {f"{m[1]}{k}" for k in range(int(m[2]), int(m[3] or m[2]) + 1)} if m else set()


def _operands(line: str) -> list[str]:
    rest = line.split(None, 1)
    return [x.strip() for x in rest[1].split(",")] if len(rest) > 1 else []


def _wait(line: str) -> int:
    """Wait states an instruction counts for."""
    return int(line.split()[1]) + 1 if line.startswith("s_nop") else 1


# wait states from a matrix instruction to the first other read of its result, on gfx950
_RESULT = (("16x16x32_bf16", 8), ("16x16x64_i8", 8), ("16x16x4_f32", 10), ("32x32x", 12))


def early_reads(lines) -> list[tuple[str, str]]:
    """Reads of a matrix instruction's result too soon behind a branch that ends its block (or behind the label that the
    block falls through to): (the instruction, the read).  Within a block the compiler keeps the distance."""
    labels = {x[:-1]: i for i, x in enumerate(lines) if x.endswith(":")}
    bad = []
    for i, line in enumerate(lines):
        m = re.match(r"s_c?branch\w* (\S+)$", line)
        ends = m or line.endswith(":")
        if not ends:
            continue
        due, states = {}, 1 if m else 0  # registers whose result is under way: states still to wait, seen from behind `line`
        for x in reversed(lines[:i]):
            if x.endswith(":") or x.startswith("s_branch") or states > 12:
                break
            if x.startswith("v_mfma"):
                need = next(n for k, n in _RESULT if k in x)
                for r in _registers(_operands(x)[0]):
                    due.setdefault(r, (need - states, x))
            states += _wait(x)
        paths = [labels[m[1]]] if m else []
        if not m or line.startswith("s_cbranch"):
            paths.append(i)
        for start in paths if due else ():
            left, passed = dict(due), 0
            for x in lines[start + 1:]:
                if x.endswith(":"):
                    continue
                if re.match(r"s_c?branch|s_endpgm", x) or passed > 12:
                    break
                ops = _operands(x)
                if not x.startswith(("v_mfma", "s_")):
                    read = ops if re.match(r"(global|flat|scratch)_store|ds_write|buffer_store", x) else ops[1:]
                    for r in set().union(*map(_registers, read)) & left.keys():
                        if left[r][0] > passed:
                            bad.append((left[r][1], x))
                for r in _registers(ops[0]) if ops else ():
                    left.pop(r, None)
                passed += _wait(x)
    return bad


def overwritten_stores(lines) -> list[tuple[str, str]]:
    """Stores of more than 8 bytes with a scalar offset register whose data the very next instruction writes again:
    the compiler leaves no wait state there, and the store has gone out with the later value."""
    code = [x for x in lines if not x.endswith(":")]
    bad = []
    for x, y in zip(code, code[1:]):
        m = re.match(r"buffer_store_dwordx[34] (v\[\d+:\d+\]), .*s\[\d+:\d+\], (s\d+|m0|vcc\w*)\b", x)
        if m and y.startswith("v_") and _operands(y) and _registers(_operands(y)[0]) & _registers(m[1]):
            bad.append((x, y))
    return bad
