// Epilogue of mx_linear, shared by the FC2 kernels it runs on:
//   out[m, n] = bf16_RNE(fn(acc + bias[group, n]) * mul[m, n] + residual[m, n])
// in fp32 on the accumulators, before their one rounding.  mul, residual and out
// are bf16 [M, N].
//
// The kernels multiply with the operands swapped (weights as the MFMA's first),
// so a lane's four accumulator elements are neighbouring columns of one row, and
// lay out the weight rows of two column tiles so that a lane's eight elements
// are eight neighbouring columns (epi_row16, epi_row32): one 16-byte access per
// operand instead of eight 2-byte ones.  (With 2-byte accesses the epilogue of
// 8192 x 4096 outputs with a residual took about 90 us more than the product.)
// N % 8 == 0, so a piece of eight columns lies within N or behind it as a whole.
//
// A piece of mul and residual is read by the thread that writes that piece of
// out, and before it does, so either may be out itself.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "copy_ring.h"
#include "gemm.h"
#include "mx_device.h"

namespace moe_mx {

// Weight row (column of out) held at row j of a tile pair.  16 x 16 MFMAs: row
// 4g + i of tile t in a pair (32 rows) is column 8g + 4t + i; 32 x 32 MFMAs: row
// 8q + 4h + i of tile t in a pair (64 rows) is column 16q + 8h + 4t + i.
__device__ __forceinline__ int epi_row16(int j) { return (j & ~31) | ((j >> 2) & 3) << 3 | ((j >> 4) & 1) << 2 | (j & 3); }
__device__ __forceinline__ int epi_row32(int j) {
  return (j & ~63) | ((j >> 3) & 3) << 4 | ((j >> 2) & 1) << 3 | ((j >> 5) & 1) << 2 | (j & 3);
}

// The epilogue's operands, read from the kernel arguments (FcArgs, the only one)
// where an epilogue begins: held from the start of a persistent kernel they would
// take scalar registers from its step loop.
__device__ __forceinline__ Epilogue epi_load() {
  const __attribute__((address_space(4))) char* args =
      (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(args));
  return *(const Epilogue*)(args + offsetof(FcArgs, epi));
}

// The lane, opaque to the compiler: what an epilogue derives from it is computed
// there, not ahead of the step loop, whose registers it would take.
__device__ __forceinline__ int epi_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// SiLU through t = exp(-|v|) <= 1, so that the tail of negative v does not pass
// through an overflowing exp(-v).  1 + t lies in [1, 2], where the reciprocal
// instruction is good to a step.
__device__ __forceinline__ float silu(float v) {
  const float t = expf(-fabsf(v));
  return v * (v < 0.0f ? t : 1.0f) * __builtin_amdgcn_rcpf(1.0f + t);
}
// GELU: v Phi(v), with Phi(-|v|) = erfc(x) / 2 at x = |v| / sqrt(2), which keeps the
// tail of negative v accurate relative to itself (1 + erf would cancel).  erfc(x) =
// exp(-x^2) t P(t), t = 1 / (1 + x/2): P is a weighted least-squares fit of degree 8 to
// erfcx(x) / t over x in [0, 14]; t P(t) with the coefficients rounded to fp32 is off by
// at most 9.8e-8 of its value (near x = 0.05).  In fp32 the result is within 7 + 2 v^2
// half steps of its value for |v| <= 13.21; there exp2's result leaves the normal
// numbers and is 0, as then is GELU of a negative v (its value: below 2^-127).
// (4674 x 7464 x 1280, E2M1 x bf16: 130 us, with erfcf 152, without a function 116.)
__device__ __forceinline__ float gelu(float v) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.35355339f, fabsf(v), 1.0f));
  float p = -5.938633031e-02f;
  p = fmaf(p, t, 2.861234119e-01f);
  p = fmaf(p, t, -4.904054181e-01f);
  p = fmaf(p, t, 2.817324350e-01f);
  p = fmaf(p, t, -2.914813096e-02f);
  p = fmaf(p, t, 2.037524415e-01f);
  p = fmaf(p, t, 2.428351139e-01f);
  p = fmaf(p, t, 2.824121019e-01f);
  p = fmaf(p, t, 2.820843310e-01f);
  const float q = 0.5f * t * p * __builtin_amdgcn_exp2f(-0.72134752f * (v * v));  // exp(-v^2 / 2)
  return v * (v < 0.0f ? q : 1.0f - q);
}
// (a comparison, not a maximum, which would turn NaN into 0)
__device__ __forceinline__ float relu2(float v) {
  const float r = v < 0.0f ? 0.0f : v;
  return r * r;
}
// (one choice for the eight values of a piece)
__device__ __forceinline__ void epi_fn(int fn, float (&v)[8]) {
  switch (fn) {
    case MX_FN_SILU:
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = silu(v[q]);
      break;
    case MX_FN_GELU:
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = gelu(v[q]);
      break;
    case MX_FN_RELU2:
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = relu2(v[q]);
      break;
    default: break;
  }
}

// bias of columns [n, n + 8) (n < N) of a group as loaded, and its values (0
// without one); loading does not wait for the data
struct EpiBias {
  uint4 lo, hi;
};
__device__ __forceinline__ EpiBias epi_bias(const Epilogue& e, int N, int group, int n) {
  EpiBias b = {};
  const int64_t i = (int64_t)group * N + n;
  if (e.bias_kind == kBiasF32) {
    const uint4* p = (const uint4*)((const float*)e.bias + i);
    b.lo = p[0];
    b.hi = p[1];
  } else if (e.bias_kind == kBiasBf16) {
    b.lo = *(const uint4*)((const uint16_t*)e.bias + i);
  } else if (e.bias_kind == kBiasF32Any) {
    const uint32_t* p = (const uint32_t*)e.bias + i;
    b.lo = make_uint4(p[0], p[1], p[2], p[3]);
    b.hi = make_uint4(p[4], p[5], p[6], p[7]);
  } else if (e.bias_kind == kBiasBf16Any) {
    const uint16_t* p = (const uint16_t*)e.bias + i;
    b.lo = make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
  }
  return b;
}
__device__ __forceinline__ float epi_bias_at(const Epilogue& e, const EpiBias& b, int q) {
  const uint32_t w[8] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, b.hi.x, b.hi.y, b.hi.z, b.hi.w};
  const bool f32 = e.bias_kind == kBiasF32 || e.bias_kind == kBiasF32Any;
  return __uint_as_float(f32 ? w[q] : q & 1 ? w[q / 2] & 0xffff0000u : w[q / 2] << 16);
}

// The second factors and residuals of the piece at element offset o
struct EpiIn {
  uint4 mul, residual;
};
__device__ __forceinline__ EpiIn epi_in(const Epilogue& e, int64_t o) {
  EpiIn in = {};
  if (e.mul) in.mul = *(const uint4*)(e.mul + o);
  if (e.residual) in.residual = *(const uint4*)(e.residual + o);
  return in;
}

// A copy wave's request for the second factors and residuals of ROWS rows by COLS
// columns from (row0, col0), cut at row_end and N, some steps before the epilogue
// reads them: a word of each 128-byte line, copied to LDS that nothing reads
// (256 bytes at lds), so that the line is in L2 by then.  (mid kernel, 2048 x 8192 x
// 2048 with a residual: 80 us against 84, 64-row tiles 104 against 111.)
template <int ROWS, int COLS>
__device__ __forceinline__ void epi_touch(const Epilogue& e, int N, int64_t row0, int64_t row_end, int col0,
                                          uint32_t lds) {
  constexpr int LINES = COLS / 64, PER = ROWS * LINES / 64;  // lines per row, words per lane
  static_assert(PER * 64 == ROWS * LINES, "whole copies");
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = 64 * i + lane;
    const int64_t row = min(row0 + j / LINES, row_end - 1);
    const int64_t o = row * N + min(col0 + 64 * (j % LINES), N - 2);
    if (e.mul) lds_copy4(e.mul + o, lds);
    if (e.residual) lds_copy4(e.residual + o, lds);
  }
}

// The piece at o from v = accumulators + bias.  FN: the function, or -1 for e.fn.
template <int FN = -1>
__device__ __forceinline__ void epi_store(const Epilogue& e, int64_t o, const EpiIn& in, float (&v)[8]) {
  const uint32_t mu[4] = {in.mul.x, in.mul.y, in.mul.z, in.mul.w};
  const uint32_t re[4] = {in.residual.x, in.residual.y, in.residual.z, in.residual.w};
  epi_fn(FN < 0 ? e.fn : FN, v);
  if (e.mul) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= __uint_as_float(q & 1 ? mu[q / 2] & 0xffff0000u : mu[q / 2] << 16);
  }
  if (e.residual) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += __uint_as_float(q & 1 ? re[q / 2] & 0xffff0000u : re[q / 2] << 16);
  }
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const v2bf o2 = {(__bf16)v[2 * q], (__bf16)v[2 * q + 1]};
    __builtin_memcpy(&w[q], &o2, 4);
  }
  *(uint4*)(e.out + o) = make_uint4(w[0], w[1], w[2], w[3]);
}

// R pieces of one row of out (row < row_end, else nothing), the first at column
// col0 and the others cstep apart; acc(q): the accumulators of piece q.  All
// loads go out before the first store, which they could not pass (out may be mul
// or residual).
template <int R, int FN = -1, class Acc>
__device__ __forceinline__ void epi_row(const Epilogue& e, int N, int64_t row, int64_t row_end, int col0, int cstep,
                                        const EpiBias (&bias)[R], Acc acc) {
  if (row >= row_end) return;
  EpiIn in[R];
#pragma unroll
  for (int q = 0; q < R; ++q)
    if (col0 + q * cstep < N) in[q] = epi_in(e, row * N + col0 + q * cstep);
#pragma unroll
  for (int q = 0; q < R; ++q)
    if (col0 + q * cstep < N) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = acc(q, i) + epi_bias_at(e, bias[q], i);
      epi_store<FN>(e, row * N + col0 + q * cstep, in[q], v);
    }
}
template <int R>
__device__ __forceinline__ void epi_biases(const Epilogue& e, int N, int group, int col0, int cstep,
                                           EpiBias (&bias)[R]) {
#pragma unroll
  for (int q = 0; q < R; ++q)
    if (col0 + q * cstep < N) bias[q] = epi_bias(e, N, group, col0 + q * cstep);
}


// P pieces whose accumulators started from the bias, `C` at a time: the loads of
// a chunk go out before the stores of the chunk before.  at(q): element offset of
// piece q, or -1 for one outside; acc(q, i): its accumulators.
template <int P, int C, int FN, class At, class Acc>
__device__ __forceinline__ void epi_pieces(const Epilogue& e, At at, Acc acc) {
  static_assert(P % C == 0, "whole chunks");
  EpiIn in[2][C];
#pragma unroll
  for (int q = 0; q < C; ++q)
    if (at(q) >= 0) in[0][q] = epi_in(e, at(q));
#pragma unroll
  for (int c = 0; c < P / C; ++c) {
    if (c + 1 < P / C) {
#pragma unroll
      for (int q = 0; q < C; ++q)
        if (at((c + 1) * C + q) >= 0) in[(c + 1) & 1][q] = epi_in(e, at((c + 1) * C + q));
    }
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int64_t o = at(c * C + q);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = acc(c * C + q, i);
      if (o >= 0) epi_store<FN>(e, o, in[c & 1][q], v);
    }
  }
}

}  // namespace moe_mx
