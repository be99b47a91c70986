"""mx4_quantize takes every size up to the documented 2^30 (the C entry point on the host, with
addresses that are never dereferenced)."""
import pytest

from tests.test_mx4_cpu import ARCH, QUANT, _call, host_only


@host_only
@pytest.mark.parametrize("size", [
    dict(batch=(1 << 23) + 1, rows=1, cols=1, ld=1, transpose=1), dict(batch=1 << 30, rows=1, cols=1, ld=1, transpose=1),
    dict(batch=1, rows=1, cols=1 << 30, ld=1 << 30, transpose=1), dict(batch=1, rows=1 << 30, cols=65, ld=65, transpose=1),
    dict(batch=3, rows=300, cols=1 << 29, ld=1 << 29, transpose=1),
    dict(batch=1, rows=1 << 30, cols=1, ld=1), dict(batch=1 << 30, rows=1, cols=1, ld=1), dict(batch=1, rows=1 << 30, cols=129, ld=129),
    dict(batch=1, rows=1, cols=1 << 30, ld=1 << 30), dict(batch=129, rows=1, cols=1 << 30, ld=1 << 30),
], ids=str)
def test_documented_sizes_pass(size):
    """They reach the check of the device."""
    assert _call("mx4_quantize", QUANT, **size) == ARCH
