"""Which kernel an mx_linear call takes: tests/linear_plan_check.cpp, compiled from
the library's own header and asked on the host."""
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple

from tests.conftest import ROOT

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
Plan = namedtuple("Plan", "kernel rows ksplit workgroups tiles workspace")
_ACT, _FMT = {"bf16": 0, "mxfp8": 1}, {"e2m1": 1, "e3m2": 2}


@functools.lru_cache(maxsize=1)
def _program():
    exe = os.path.join(tempfile.mkdtemp(prefix="linear_plan"), "linear_plan_check")
    src = os.path.join(ROOT, "tests", "linear_plan_check.cpp")
    subprocess.run([HIPCC, "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "block_scaled_precision_amd", "csrc"), src, "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def plans(problems):
    """Plans of problems (M, N, K, groups, fmt, act) with bf16 rows as given; None for
    one that is not supported."""
    text = "\n".join(f"{M} {N} {K} {G} {_ACT[act]} {_FMT[fmt]} 0" for M, N, K, G, fmt, act in problems)
    r = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True, timeout=120)
    out = []
    for line in r.stdout.splitlines():
        f = line.split()
        out.append(None if f == ["unsupported"] else Plan(f[0], *map(int, f[1:])))
    assert len(out) == len(problems)
    return out
