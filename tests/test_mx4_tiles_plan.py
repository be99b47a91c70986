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


def test_lists_of_256_row_tiles():
    from tests import test_gpu_mx4_tiles as t
    problems = [(M, N, K, G, codes) for M, N, K in t.SCALED for G in (0, 5) for codes in (False, True)]
    problems += [(sum(c) + 5, N, K, len(c), codes) for N, K, c in t.COUNTS for codes in (False, True)]
    problems += [(M, N, K, 4, False) for M, N, K in t.OUT_OF_ORDER]
    problems += [(M, N, K, G, True) for M, N, K, G in t.ALIGNED]
    wrong = [(q, p) for q, p in zip(problems, plans(problems)) if (p.kernel, p.rows) != ("tile", 256)]
    assert not wrong, wrong
    for some in ([(M, N, K, G, True) for M, N, K, G in t.IN_PLACE], t.AT_ONCE):
        assert [p.rows for p in plans(some)] == [256] * (len(some) - 1) + [128], some


def test_every_list_meets_every_tile_height():
    """The shapes of each check in both files together."""
    from tests import test_gpu_mx4_linear as lin
    from tests import test_gpu_mx4_tiles as t
    lists = {
        "scales": [(M, N, K, G, True) for M, N, K in lin.PICKED + t.SCALED for G in (0, 5)],
        "biases": [(M, N, K, G, True) for M, N, K, G in t.ALIGNED + [(3, 72, 256, 0), (300, 2056, 640, 0), (3000, 4104, 512, 0)]],
        "at once": lin.AT_ONCE + t.AT_ONCE,
        "functions": [(M, N, K, G, False) for _, _, M, N, K, G in lin.SOME + t.LARGE],
    }
    for name, problems in lists.items():
        got = {p.rows for p in plans(problems) if p.kernel in ("tile", "ranges")}
        assert got == {64, 128, 256}, (name, got)
