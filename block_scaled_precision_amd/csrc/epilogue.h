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

}  // namespace moe_mx
