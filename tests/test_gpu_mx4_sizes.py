"""mx4_quantize of more work than one launch holds (2^23 workgroups), against the same rows in a
small call."""
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

PERIOD = 1000


def _repeats(got, part, what):
    """Rows of got are those of part over and over."""
    step = PERIOD << 14
    whole = part.repeat(step // PERIOD, 1)
    for i in range(0, got.shape[0], step):
        own = got[i:i + step]
        assert torch.equal(own, whole[:own.shape[0]]), f"{what} from {i}"


@pytest.fixture
def memory():
    yield
    torch.cuda.empty_cache()


def _values(n):
    """PERIOD values and bytes, and n that repeat them."""
    x = gen.normal((PERIOD,), 3, 90).to(torch.bfloat16).cuda()
    random = gen.random_bytes((PERIOD,), 3, 91).cuda()
    times = -(-n // PERIOD)
    return x, random, x.repeat(times)[:n], random.repeat(times)[:n]


def test_many_small_matrices(memory):
    from block_scaled_precision_amd import moe_mx as m
    n = (1 << 24) + 77  # three launches
    print_flush(f"mx4_quantize transposed {n} matrices")
    x, random, many, bytes_ = _values(n)
    for rnd, all_rnd in ((None, None), (random.view(-1, 1, 1), bytes_.view(-1, 1, 1))):
        codes, scales = m.mx4_quantize(many.view(-1, 1, 1), transpose=True, random=all_rnd)
        c, s = m.mx4_quantize(x.view(-1, 1, 1), transpose=True, random=rnd)
        _repeats(codes.view(n, -1), c.view(PERIOD, -1), "codes")
        _repeats(scales.view(n, -1), s.view(PERIOD, -1), "scales")


@pytest.mark.parametrize("transpose", [True, False])
def test_many_columns_and_rows(transpose, memory):
    """One row of 2^29 columns, transposed, and as many rows of one column."""
    from block_scaled_precision_amd import moe_mx as m
    n = (1 << 29) + 77
    print_flush(f"mx4_quantize transpose={transpose} {n} vectors")
    x, random, many, bytes_ = _values(n)
    shape = (lambda t: t.view(1, -1)) if transpose else (lambda t: t.view(-1, 1))
    codes, scales = m.mx4_quantize(shape(many), transpose=transpose, random=shape(bytes_))
    c, s = m.mx4_quantize(shape(x), transpose=transpose, random=shape(random))
    assert codes.shape == (n, 64) and scales.shape == (n, 4)
    _repeats(codes, c, "codes")
    _repeats(scales, s, "scales")
