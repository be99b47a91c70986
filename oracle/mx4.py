"""MXFP4 operands: blocks of 32 along a matrix's rows or columns, rotated and
stochastically rounded on request, and the product of two operands -- oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Sources.  "TokenSpeed SiTU" page, section "Supported contract" (``MxE2m1``), and
"mxfp6-sm120" page, section "Execution model" (a UE8M0 scale per 32 K values, dynamic
quantization).  The nearest rounding is ``oracle.mx.quantize``.  The rest is on no
page: a rotation by the 32-point Hadamard matrix with signs, which the fp32 result of
each sum in a fixed order defines (numpy's float32 here), and a rounding that takes
the upper neighbour with the probability of the position between the two.
"""
from __future__ import annotations

import numpy as np

from . import gemm, mx

K_STEP = 128  # operands end at a multiple of this, with zeros


def rotate(v: np.ndarray, signs: np.ndarray) -> np.ndarray:
    """Blocks [..., 32] of fp32 values rotated, every operation rounded to fp32."""
    v = (v.astype(np.float32) * signs.astype(np.float32)).astype(np.float32)
    for d in (1, 2, 4, 8, 16):
        out = np.empty_like(v)
        for i in range(32):
            j = i ^ d
            out[..., i] = v[..., i] + v[..., j] if i < j else v[..., j] - v[..., i]
        v = out
    return v * np.float32(32 ** -0.5)


def round_stochastically(v: np.ndarray, random: np.ndarray):
    """(codes, scales) of blocks [..., 32] with one byte per value."""
    table = mx.decode_table("e2m1")[:8]
    amax = np.max(np.abs(v), axis=-1)
    _, ex = np.frexp(amax)
    s = np.clip(ex - 3, -127, 127)
    s = np.where(amax > 6 * np.ldexp(1.0, s), s + 1, s)
    s = np.where(amax < 2.0 ** -126, -127, s)
    q = np.abs(np.ldexp(v, -s[..., None]))
    lo = np.clip(np.searchsorted(table, q, side="right") - 1, 0, 6)
    part = (q - table[lo]) / (table[lo + 1] - table[lo])
    code = lo + (part * 256 - random > 0.5)
    return (code | np.signbit(v).astype(np.int64) << 3).astype(np.uint8), (s + 127).astype(np.uint8)


def operand(src: np.ndarray, transpose: bool = False, signs=None, random=None):
    """Packed codes [..., rows, K/2] and scales [..., rows, K/32] of src [..., R, C]."""
    v = np.asarray(src, dtype=np.float64)
    if transpose:
        v = np.swapaxes(v, -1, -2)
        random = None if random is None else np.swapaxes(random, -1, -2)
    pad = [(0, 0)] * (v.ndim - 1) + [(0, -v.shape[-1] % K_STEP)]
    v = np.pad(v, pad)
    blocks = v.reshape(v.shape[:-1] + (-1, mx.BLOCK))
    over = np.zeros(blocks.shape[:-1], dtype=bool)
    if signs is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            blocks = rotate(blocks, signs).astype(np.float64)
        over = ~np.isfinite(blocks).all(-1)  # left fp32: the NaN scale, codes unspecified
        blocks[over] = 0.0
    if random is None:
        codes, scales = mx.quantize(blocks.reshape(v.shape), "e2m1")
    else:
        codes, scales = round_stochastically(blocks, np.pad(random, pad).reshape(blocks.shape).astype(np.int64))
    return mx.pack(codes.reshape(v.shape), "e2m1"), np.where(over, 255, scales).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values that packed codes stand for."""
    return mx.dequantize(mx.unpack(codes, "e2m1", 2 * codes.shape[-1]), scales, "e2m1")


def mx4_linear(a, w_packed, w_scale, *, a_scale=None, **kw):
    """oracle.gemm.mx_linear with a [M, K] quantized to E2M1 first, or given as packed codes
    [M, K/2] with a_scale [M, K/32]."""
    if a_scale is None:
        a, a_scale = operand(a)
    return gemm.mx_linear(values(a, a_scale), w_packed, w_scale, wfmt="e2m1", act="bf16", **kw)
