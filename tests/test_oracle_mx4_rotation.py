"""The oracle's rotation at the end of fp32's range."""
import numpy as np
import pytest

from oracle import mx4


@pytest.mark.parametrize("random", [False, True])
def test_a_block_that_leaves_fp32_has_the_nan_scale(random):
    signs = np.where(np.arange(32) % 3 == 0, -1.0, 1.0)
    below = float(np.nextafter(np.float32(2.0 ** 123), np.float32(0)))
    src = np.zeros((4, 128))
    src[0] = np.tile(signs, 4) * below        # one sum of 32 equal values, which fp32 still holds
    src[1, 32:64] = signs * 2.0 ** 123        # one step more
    src[2, 5] = np.finfo(np.float32).max      # alone it stays
    src[3, 64:66] = np.finfo(np.float32).max  # 2 (or 0) times it does not
    r = np.full(src.shape, 100) if random else None
    codes, scales = mx4.operand(src, signs=signs, random=r)
    assert np.argwhere(scales == 255).tolist() == [[1, 1], [3, 2]]
    v = mx4.values(codes, scales)
    total = np.abs(v[0, :32]).max()
    # 32 values / sqrt(32), to within the rounding to a code (a sixth, or up to 6 of 8)
    assert abs(total / (below * 32 ** 0.5) - 1) <= 0.25 and not v[0, 1:32].any()
    assert np.isnan(v[1, 32:64]).all() and np.isfinite(np.delete(v[1], np.s_[32:64])).all()
    assert np.isfinite(v[2]).all()


def test_smaller_blocks_are_as_they_were():
    rng = np.random.default_rng(1)
    src, signs = rng.normal(size=(8, 256)).astype(np.float32), rng.choice([-1.0, 1.0], 32)
    codes, scales = mx4.operand(src, signs=signs)
    v = mx4.rotate(src.astype(np.float64).reshape(8, 8, 32), signs).reshape(8, 256)
    want = mx4.mx.quantize(v.astype(np.float64), "e2m1")
    assert np.array_equal(codes, mx4.mx.pack(want[0], "e2m1")) and np.array_equal(scales, want[1])
