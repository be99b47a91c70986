"""The shapes of tests/test_gpu_mx4_tiles.py take the kernels they name (no GPU needed)."""
import os

import pytest

from tests.linear_plan import HIPCC
from tests.mx4_plan import plans

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")


def test_functions_run_on_the_tiles_they_name():
    from tests.test_gpu_mx4_tiles import LARGE
    got = plans([(M, N, K, G, False) for _, _, M, N, K, G in LARGE])
    wrong = [(c, p) for c, p in zip(LARGE, got) if (p.kernel, p.rows) != c[:2]]
    assert not wrong, wrong
    for rows in (128, 256):
        for grouped in (False, True):
            own = [c for c in LARGE if c[1] == rows and (c[5] > 0) == grouped]
            # stages of 256 K even and odd in number, the last one whole and half
            stages = {(-(-c[4] // 256) % 2, c[4] % 256) for c in own}
            assert len({s[0] for s in stages}) == 2 and len({s[1] for s in stages}) == 2, own
            # several items for a workgroup, and at most one
            items = [-(-c[2] // rows) * -(-c[3] // 256) for c in own]
            assert max(items) > 256 > min(items), own
