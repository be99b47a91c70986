// Epilogue of mx_linear, shared by the FC2 kernels it runs on:
//   out[m, n] = bf16_RNE(fn(acc + bias[group, n]) * mul[m, n] + residual[m, n])
// in fp32 on the accumulators, before their one rounding.  A kernel's lanes
// hold accumulators of fixed columns, so each column's bias is loaded once per
// item; mul, residual and out are bf16 [M, N].  An element of mul and residual
// is read by the thread that writes that element of out, and before it does,
// so either may be out itself.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"
#include "mx_device.h"

namespace moe_mx {

// bias of column n (< N) of a group, 0 without one
__device__ __forceinline__ float epi_bias(const FcArgs& p, int group, int n) {
  if (!p.epi.bias) return 0.f;
  const int64_t i = (int64_t)group * p.N + n;
  return p.epi.bias_bf16 ? bf16_bits_to_f32(((const uint16_t*)p.epi.bias)[i]) : ((const float*)p.epi.bias)[i];
}

// SiLU through t = exp(-|v|) <= 1, so that the tail of negative v does not pass
// through an overflowing exp(-v); erfc rather than 1 + erf: for negative v the sum would cancel, leaving an
// error relative to v instead of to the result
__device__ __forceinline__ float epi_fn(int fn, float v) {
  switch (fn) {
    case MX_FN_SILU: {
      const float t = expf(-fabsf(v));
      return v * (v < 0.0f ? t : 1.0f) / (1.0f + t);
    }
    case MX_FN_GELU: return 0.5f * v * erfcf(-0.70710678f * v);
    case MX_FN_RELU2: {
      const float r = fmaxf(v, 0.0f);
      return r * r;
    }
    default: return v;
  }
}

// out[o] from v = acc + bias (o: element offset of (m, n))
__device__ __forceinline__ void epi_store(const FcArgs& p, int64_t o, float v) {
  v = epi_fn(p.epi.fn, v);
  if (p.epi.mul) v *= bf16_bits_to_f32(p.epi.mul[o]);
  if (p.epi.residual) v += bf16_bits_to_f32(p.epi.residual[o]);
  ((__bf16*)p.obuf)[o] = (__bf16)v;
}

// R rows from row0 (rows from row_end on: none) by C columns col0, col0 +
// cstep, ... of out, v(i, n) their accumulators.  The block's second factors and
// residuals are loaded before its first store: a store may alias them, so the
// loads of a row could not pass the stores of the row before, and each would
// cost a memory latency.  FN: the function, or -1 to take it from p.
template <int R, int C, int FN = -1, class V>
__device__ __forceinline__ void epi_block(const FcArgs& p, int group, int64_t row0, int64_t row_end, int col0,
                                          int cstep, V v) {
  float bias[C];
  uint16_t mu[R][C], re[R][C];
#pragma unroll
  for (int n = 0; n < C; ++n) bias[n] = col0 + n * cstep < p.N ? epi_bias(p, group, col0 + n * cstep) : 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < C; ++n) {
      const int col = col0 + n * cstep;
      const bool in = row0 + i < row_end && col < p.N;
      const int64_t o = (row0 + i) * p.N + col;
      mu[i][n] = p.epi.mul && in ? p.epi.mul[o] : 0;
      re[i][n] = p.epi.residual && in ? p.epi.residual[o] : 0;
    }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < C; ++n) {
      const int col = col0 + n * cstep;
      if (row0 + i >= row_end || col >= p.N) continue;
      float x = epi_fn(FN < 0 ? p.epi.fn : FN, v(i, n) + bias[n]);
      if (p.epi.mul) x *= bf16_bits_to_f32(mu[i][n]);
      if (p.epi.residual) x += bf16_bits_to_f32(re[i][n]);
      ((__bf16*)p.obuf)[(row0 + i) * p.N + col] = (__bf16)x;
    }
}

}  // namespace moe_mx
