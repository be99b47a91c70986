"""The choice of mx4_linear's kernel, on the host (no GPU needed)."""
import os

import pytest

from tests.linear_plan import HIPCC
from tests.mx4_plan import plans

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
SIZES = [(M, N, K, G) for M in (1, 16, 100, 5000, 10 ** 6, 1 << 24, 1 << 27, 1 << 30)
         for N in (8, 24, 136, 4096, 16384, 1 << 23) for K in (128, 384, 512, 896, 7168, 1 << 24) for G in (0, 1, 8, 1024)
         if M * N <= 1 << 35 and M * N * K <= 1 << 52]


@pytest.mark.parametrize("codes", [False, True])
def test_every_choice_fits_its_launch(codes):
    problems = [(M, N, K, G, codes) for M, N, K, G in SIZES]
    for (M, N, K, G, _), plan in zip(problems, plans(problems)):
        if plan.kernel == "few":  # a workgroup of 512 threads per item, fewer than 2^32 threads
            tiles = plan.tiles if G else -(-M // 16)
            assert 0 < tiles * -(-N // 16) <= 1 << 20, (M, N, K, G, plan)
        if plan.kernel == "tile":
            assert K >= 512 and N <= 1 << 22, (M, N, K, G, plan)
        # nothing needs more than the codes twice over, the tile list and the partial sums
        assert plan.workspace <= 2 * M * K + 64 * (M + 1024) + (1 << 20) + 64 * M * N, (M, N, K, G, plan)


def test_kernel_cases_take_the_kernels_they_name():
    from tests.test_gpu_mx4_linear import CASES
    for codes in (False, True):
        got = plans([(M, N, K, G, codes) for _, _, M, N, K, G in CASES])
        wrong = [(c, p) for c, p in zip(CASES, got) if (p.kernel, p.rows) != c[:2]]
        assert not wrong, wrong


def test_kernel_cases_cover_every_choice():
    """Every kernel and tile height that a broad grid of sizes chooses, with or without
    groups, has a case; tiles also one with K % 256 != 0, one with more items than
    workgroups and N % 256 != 0."""
    from tests.test_gpu_mx4_linear import CASES
    covered = {(k, r, G > 0) for k, r, M, N, K, G in CASES}
    grid = [(M, N, K, G, c) for M in (1, 16, 48, 100, 300, 520, 900, 1900, 4200, 9000, 20000) for N in
            (8, 264, 1032, 2056, 4096, 8200) for K in (128, 640, 1024, 2048, 7168) for G in (0, 5, 64) for c in (0, 1)]
    for (M, N, K, G, c), p in zip(grid, plans(grid)):
        assert (p.kernel, p.rows, G > 0) in covered, (p, M, N, K, G, c)
    for kernel, rows, grouped in covered:
        if kernel != "tile":
            continue
        own = [c for c in CASES if c[:2] == (kernel, rows) and (c[5] > 0) == grouped]
        assert any(c[4] % 256 for c in own) and any(c[3] % 256 for c in own), own
        assert any(-(-c[2] // rows) * -(-c[3] // 256) > 256 for c in own), own
