"""Pins for the MXFP4 operand oracle (CPU only)."""
import numpy as np
import pytest
import scipy.linalg

from oracle import gemm as og
from oracle import mx, mx4


def test_rotation_is_the_hadamard_matrix():
    """Against scipy's matrix in float64: five sums of two and a product, each off by half
    a step of a sum of at most 32 magnitudes; and it keeps products."""
    rng = np.random.default_rng(0)
    h = scipy.linalg.hadamard(32) / np.sqrt(32)
    signs = np.where(rng.random(32) < 0.5, -1.0, 1.0)
    v = rng.standard_normal((50, 32)).astype(np.float32)
    ref = (v.astype(np.float64) * signs) @ h
    got = mx4.rotate(v, signs).astype(np.float64)
    assert np.all(np.abs(got - ref) <= 7 * 2.0 ** -24 * np.abs(v).sum(1, keepdims=True) / np.sqrt(32))
    assert np.allclose(got @ got.T, v.astype(np.float64) @ v.T.astype(np.float64), atol=1e-4)


def test_integers_rotate_exactly():
    v = np.arange(-16, 16, dtype=np.float32)[None]
    signs = np.ones(32)
    exact = v.astype(np.float64) @ scipy.linalg.hadamard(32)
    assert np.array_equal(mx4.rotate(v, signs), (exact * np.float32(32 ** -0.5)).astype(np.float32))


@pytest.mark.parametrize("q,part", [(0.0, 0.0), (0.125, 0.25), (0.5, 0.0), (1.75, 0.5), (2.25, 0.25), (3.5, 0.5),
                                    (4.5, 0.25), (5.0, 0.5), (5.9375, 0.96875), (6.0, 0.0)])
def test_rounding_probabilities(q, part):
    """Over all 256 bytes the upper neighbour comes up 256 * part times: the mean is q."""
    v = np.zeros((256, 32))
    v[:, 0], v[:, 1], v[:, 2] = 6.0, q, -q  # 6 keeps the scale at 1
    codes, scales = mx4.round_stochastically(v, np.arange(256)[:, None] * np.ones((1, 32), dtype=np.int64))
    assert (scales == 127).all()
    vals = mx.decode(codes, "e2m1")
    table = mx.decode_table("e2m1")[:8]
    assert (vals[:, 1] > q).sum() == round(256 * part) if part else (vals[:, 1] == q).all()
    assert vals[:, 1].mean() == q and vals[:, 2].mean() == -q and set(vals[:, 1]) <= set(table)


@pytest.mark.parametrize("amax,scale", [(6.0, 127), (6.0000005, 128), (4.0, 127), (8.0, 128), (12.0, 128), (12.5, 129),
                                        (0.0, 0), (2.0 ** -126, 0), (1.75 * 2.0 ** -126, 0), (2.0 ** -140, 0),
                                        (1.75 * 2.0 ** -124, 2), (1.5 * 2.0 ** -124, 1), (1.75 * 2.0 ** 127, 253)])
def test_nothing_saturates_with_random_bytes(amax, scale):
    v = np.full((1, 32), np.float32(amax), dtype=np.float64)
    for r in (0, 255):
        codes, scales = mx4.round_stochastically(v, np.full((1, 32), r))
        assert scales[0] == scale
        vals = mx.dequantize(codes, scales, "e2m1")
        step = 2 * 2.0 ** (float(scale) - 127)
        assert np.all(np.abs(vals - v) < step)


def test_operand_layout():
    """Along rows it is the padded matrix quantized; transposed, the transpose's; a block of
    the padding is zero."""
    rng = np.random.default_rng(2)
    src = rng.standard_normal((70, 45)).astype(np.float32)
    codes, scales = mx4.operand(src)
    assert codes.shape == (70, 64) and scales.shape == (70, 4) and (scales[:, 2:] == 0).all()
    c, s = mx.quantize(np.pad(src.astype(np.float64), ((0, 0), (0, 83))), "e2m1")
    assert np.array_equal(codes, mx.pack(c, "e2m1")) and np.array_equal(scales, s)
    tc, ts = mx4.operand(src, transpose=True)
    rc, rs = mx4.operand(np.ascontiguousarray(src.T))
    assert np.array_equal(tc, rc) and np.array_equal(ts, rs) and tc.shape == (45, 64)
    r = rng.integers(0, 256, src.shape)
    for signs in (None, np.where(rng.random(32) < 0.5, -1.0, 1.0)):
        a = mx4.operand(src, True, signs, r)
        b = mx4.operand(np.ascontiguousarray(src.T), False, signs, np.ascontiguousarray(r.T))
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
    vals = mx4.values(*mx4.operand(src))
    assert np.abs(vals[:, :45] - src).max() <= np.abs(src).max() / 4 and (vals[:, 45:] == 0).all()


def test_gradients_are_products_of_transposed_operands():
    """With operands that E2M1 holds exactly, dX = dY W and dW = dY^T X come out exactly."""
    rng = np.random.default_rng(3)
    table = np.array([0, 0.5, 1, 2, 4, 6, -1, -3])

    def exact(*shape):
        v = rng.choice(table, shape)
        v[:] = np.where(rng.random(shape) < 0.2, 6.0, v)
        return v
    dy, x, w = exact(96, 40), exact(96, 24), exact(40, 24)
    for blocks in (dy, x, w):  # a 4 or 6 in every block, so that all scales are 1
        blocks[::8] = 6.0
        blocks[:, ::8] = 6.0
    dx, _, _ = mx4.mx4_linear(*(mx4.operand(dy)[0], *mx4.operand(w, transpose=True)), a_scale=mx4.operand(dy)[1])
    assert np.array_equal(dx, dy @ w)
    g = mx4.operand(dy, transpose=True)
    dw, _, _ = mx4.mx4_linear(g[0], *mx4.operand(x, transpose=True), a_scale=g[1])
    assert np.array_equal(dw, dy.T @ x)


def test_product_is_the_linear_oracle_on_decoded_values():
    rng = np.random.default_rng(4)
    a, w = rng.standard_normal((5, 128)), rng.standard_normal((8, 128))
    wc, ws = mx4.operand(w)
    ref, _, _ = og.mx_linear(mx4.values(*mx4.operand(a)), wc, ws, wfmt="e2m1", act="bf16", fn="silu")
    got, _, _ = mx4.mx4_linear(a, wc, ws, fn="silu")
    codes, scales = mx4.operand(a)
    given, _, _ = mx4.mx4_linear(codes, wc, ws, a_scale=scales, fn="silu")
    assert np.array_equal(got, ref) and np.array_equal(given, ref)
