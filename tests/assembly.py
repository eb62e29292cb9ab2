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
