"""Launch shapes of moe_balance and its gradient, on the host (no GPU needed): the library's own
header, compiled by tests/balance_plan_check.cpp."""
import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.linear_plan import HIPCC

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
TOKENS = [0, 1, 16, 128, 129, 4096, 8191, 65536, 100_003, 1 << 20, (1 << 24) + 1, 1 << 27, 1 << 29, (1 << 29) + 1, (1 << 30) - 1, 1 << 30]
EXPERTS = [1, 8, 33, 36, 64, 65, 127, 128, 256, 384, 1000, 1023, 1024]
SEQUENCES = [1, 2, 4, 5, 13, 1024, 64_500, 65_536, 1 << 17, 1 << 20]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("balance_plan") / "balance_plan_check")
    subprocess.run([HIPCC, "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "block_scaled_precision_amd", "csrc"),
                    os.path.join(ROOT, "tests", "balance_plan_check.cpp"), "-o", exe], check=True, capture_output=True)
    sizes = [(T, E, S) for T in TOKENS for E in EXPERTS for S in SEQUENCES]
    r = subprocess.run([exe], input="\n".join("%d %d %d" % s for s in sizes), capture_output=True, text=True, check=True,
                       timeout=60)
    lines = r.stdout.splitlines()
    assert len(lines) == len(sizes)
    return [(s, None if line == "unsupported" else [int(v) for v in line.split()]) for s, line in zip(sizes, lines)]


def test_every_launch_has_fewer_than_2_32_threads(plans):
    for (T, E, S), plan in plans:
        if S * E > 1 << 27:
            assert plan is None
            continue
        chunks, rows, finish, _, *grad = plan
        assert max(chunks, 1) * 256 < 1 << 32 and finish * 1024 < 1 << 32, (T, E, S, plan)
        for per, blocks in (grad[:2], grad[2:])[:1 if E % 4 else 2]:
            assert blocks * 256 < 1 << 32 and blocks * per >= T, (T, E, S, plan)
            assert blocks == 0 or (blocks - 1) * per < T, (T, E, S, plan)


def test_chunks_cover_the_rows_and_stay_short(plans):
    for (T, E, S), plan in plans:
        if plan is None or plan[3] == 0:
            continue
        chunks, rows, _, workspace = plan[:4]
        assert chunks * rows >= T and rows <= 256
        # sums of p and counts of every chunk and sequence, and what else there is
        assert workspace >= (chunks + S) * (8 * E + 8) + 8 * S
        assert workspace <= (chunks + S) * (8 * E + 8) + S * (E + 64) + 4096
