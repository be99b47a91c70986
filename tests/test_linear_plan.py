"""The choice of mx_linear's kernel, on the host (no GPU needed)."""
import os

import pytest

from tests.linear_plan import HIPCC, plans

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
TYPES = [(f, a) for f in ("e2m1", "e3m2") for a in ("bf16", "mxfp8")]
# rows and columns of 2 to 2^30 and 8 to 2^14, products within the documented limits
SIZES = [(M, N, K, G) for M in (1, 16, 100, 5000, 10 ** 6, 1 << 24, 1 << 27, 1 << 30)
         for N in (8, 24, 40, 136, 4096, 16384) for K in (128, 896, 7168) for G in (0, 1, 8, 1024)
         if M * N <= 1 << 35 and M * N * K <= 1 << 52]


@pytest.mark.parametrize("fmt,act", TYPES)
def test_every_choice_fits_its_launch(fmt, act):
    """The few-row kernel's grid has a workgroup of 512 threads per item, and a launch
    holds fewer than 2^32 threads."""
    problems = [(M, N, K, G, fmt, act) for M, N, K, G in SIZES]
    for problem, plan in zip(problems, plans(problems)):
        assert plan.kernel != "none", problem
        if plan.kernel == "few":
            assert 0 < plan.workgroups <= 1 << 20, f"{problem}: {plan.workgroups} workgroups"


def test_kernel_cases_take_the_kernels_they_name():
    from tests.test_gpu_linear_kernels import CASES
    got = plans([(M, N, K, G, fmt, act) for _, _, _, M, N, K, G, fmt, act in CASES])
    wrong = [(c, p) for c, p in zip(CASES, got) if (p.kernel, p.rows, p.ksplit > 1) != c[:3]]
    assert not wrong, wrong


def test_kernel_cases_cover_every_choice():
    """Every kernel, tile height and K split that a broad grid of sizes chooses, of
    each weight format, activation type and with or without groups, has a case; mid
    and tiled also one with K % 512 != 0, and each large-tile kernel one with more items
    than there are workgroups and N % 256 != 0."""
    from tests.test_gpu_linear_kernels import CASES
    covered = {(k, r, s, G > 0, f, a) for k, r, s, M, N, K, G, f, a in CASES}
    grid = [(M, N, K, G) for M in (1, 16, 48, 100, 300, 520, 900, 1900, 4200, 9000, 20000) for N in
            (8, 264, 1032, 2056, 4096, 4160, 8200) for K in (128, 640, 1024, 2048, 3712, 7168) for G in (0, 5, 64)]
    for fmt, act in TYPES:
        problems = [(M, N, K, G, fmt, act) for M, N, K, G in grid]
        for (M, N, K, G, _, _), p in zip(problems, plans(problems)):
            assert (p.kernel, p.rows, p.ksplit > 1, G > 0, fmt, act) in covered, (p, M, N, K, G, fmt, act)
    cols = {("mid", 64): 256, ("mid", 128): 256, ("tiled", 128): 256, ("tiled", 192): 128, ("wide", 192): 256}
    for kernel, rows, split, grouped, fmt, act in covered:
        if (kernel, rows) not in cols:
            continue
        own = [c for c in CASES if c[:3] == (kernel, rows, split) and (c[6] > 0) == grouped and c[7:] == (fmt, act)]
        assert any(-(-c[3] // rows) * -(-c[4] // cols[kernel, rows]) > 256 for c in own), own
        assert any(c[4] % 256 for c in own), own
    for kernel in ("mid", "tiled"):
        for fmt, act in TYPES:
            own = [c for c in CASES if c[0] == kernel and c[7:] == (fmt, act)]
            assert not own or any(c[5] % 512 for c in own), (kernel, fmt, act)


def test_long_cases_take_the_kernels_they_name():
    from tests.test_gpu_linear_kernels import LONG
    got = plans([c[1:] for c in LONG])
    assert [p.kernel for p in got] == [c[0] for c in LONG]
