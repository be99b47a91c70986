"""Dense MX GEMM with bf16 output -- oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Sources.
* "mxfp6-sm120" page, table of paths, "Dense" row: a shape-aware W6A8 GEMM
  for linear, attention and MLP projections.
* Same page, section "Execution model" (figure): FP16/BF16 activations are
  quantized dynamically to E4M3 with one UE8M0 scale per 32 K values; the
  weight is packed MX with one UE8M0 scale per 32 K values; the block-scaled
  products accumulate in FP32 and the output is FP16/BF16.
* Same page, section "Dense GEMM and MoE layer": the dense outputs were
  compared exactly against a matmul of the decoded operands.
* Same page, section "Validated scope", "Dense GEMM" row: M > 0, N % 8 == 0,
  K % 128 == 0.

Readings (the plainest ones): C[m, n] = alpha * sum_k A'[m, k] * W'[n, k],
where W' is the decoded MX weight [N, K] and A' is either the bf16 values of
A (bf16 activations: the W4A16 form of the layer's own FC GEMMs) or A
quantized to MXFP8 along K and decoded (the W4A8 / W6A8 form); A may also be
given already quantized (E4M3 codes + E8M0 scales).  The result is float64;
the device returns one bf16 rounding (round half to even) of its fp32
accumulation, so wherever that accumulation is exact the two agree bit for
bit after rounding this result to bf16.

``mx_linear`` adds the epilogue of a linear layer (bias, activation, product
with a second operand, residual) and groups of rows with a matrix each.
"""
from __future__ import annotations

import math

import numpy as np

from . import mx
from .moe import activations, decode_weight


def mx_gemm(a, w_packed, w_scale, *, wfmt: str, act: str, alpha: float = 1.0, a_scale=None) -> np.ndarray:
    """a [M, K] exact bf16 values (float64), or E4M3 codes (uint8) when
    ``a_scale`` [M, K/32] is given; w_packed [N, K*bits/8] + w_scale [N, K/32]
    in ``wfmt`` ("e2m1" | "e3m2"); act "bf16" | "mxfp8".  Returns C [M, N]
    float64."""
    if a_scale is not None:
        if act != "mxfp8":
            raise ValueError("pre-quantized activations are MXFP8")
        A = mx.dequantize(np.asarray(a, dtype=np.uint8), a_scale, "e4m3")
    else:
        A = activations(np.asarray(a, dtype=np.float64), act)
    K = A.shape[1]
    W = decode_weight(w_packed, w_scale, wfmt, K)
    return alpha * (A @ W.T)


def linear_fn(v: np.ndarray, fn: str) -> np.ndarray:
    if fn == "none":
        return v
    if fn == "silu":
        return v / (1.0 + np.exp(-v))
    if fn == "gelu":  # v times the normal distribution function at v
        return v * np.vectorize(lambda z: 0.5 * math.erfc(-z / math.sqrt(2.0)), otypes=[np.float64])(v)
    if fn == "relu2":
        return np.maximum(v, 0.0) ** 2
    raise ValueError(fn)


def mx_linear(a, w_packed, w_scale, *, wfmt: str, act: str, bias=None, fn: str = "none", mul=None, residual=None,
              offsets=None, a_scale=None):
    """(out, sum over k of |a w|, v) in float64 [M, N]; with offsets [G + 1], w,
    w_scale and bias have a leading axis of G and rows [offsets[g] - offsets[0],
    offsets[g+1] - offsets[0]) take entry g; rows of no group are NaN."""
    M = a.shape[0]
    if offsets is None:
        w_packed, w_scale = w_packed[None], w_scale[None]
        bias = None if bias is None else bias[None]
        offsets = [0, M]
    N = w_packed.shape[1]
    out, size, v_all = (np.full((M, N), np.nan) for _ in range(3))
    if a_scale is not None:
        A = mx.dequantize(np.asarray(a, dtype=np.uint8), a_scale, "e4m3")
    else:
        A = activations(np.asarray(a, dtype=np.float64), act)
    for g in range(len(offsets) - 1):
        rows = slice(int(offsets[g] - offsets[0]), int(offsets[g + 1] - offsets[0]))
        if rows.start == rows.stop:
            continue
        W = decode_weight(w_packed[g], w_scale[g], wfmt, A.shape[1])
        v = A[rows] @ W.T + (0.0 if bias is None else bias[g])
        size[rows] = np.abs(A[rows]) @ np.abs(W).T
        v_all[rows] = v
        out[rows] = linear_fn(v, fn) * (1.0 if mul is None else mul[rows]) + (0.0 if residual is None else residual[rows])
    return out, size, v_all
