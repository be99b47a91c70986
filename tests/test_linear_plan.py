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
