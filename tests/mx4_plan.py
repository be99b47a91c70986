"""Which kernel an mx4_linear call takes: tests/mx4_plan_check.cpp, compiled from the
library's own header and asked on the host."""
import functools
import os
import subprocess
import tempfile
from collections import namedtuple

from tests.conftest import ROOT
from tests.linear_plan import HIPCC

Plan = namedtuple("Plan", "kernel rows tiles workspace")


@functools.lru_cache(maxsize=1)
def _program():
    exe = os.path.join(tempfile.mkdtemp(prefix="mx4_plan"), "mx4_plan_check")
    src = os.path.join(ROOT, "tests", "mx4_plan_check.cpp")
    subprocess.run([HIPCC, "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "block_scaled_precision_amd", "csrc"), src, "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def plans(problems):
    """Plans of problems (M, N, K, groups, codes given); None for one that is not supported."""
    text = "\n".join(f"{M} {N} {K} {G} {int(codes)}" for M, N, K, G, codes in problems)
    r = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True, timeout=120)
    out = []
    for line in r.stdout.splitlines():
        f = line.split()
        out.append(None if f == ["unsupported"] else Plan(f[0], *map(int, f[1:])))
    assert len(out) == len(problems)
    return out
