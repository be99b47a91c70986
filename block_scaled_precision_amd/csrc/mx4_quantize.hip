// MXFP4 operands: mx4_quantize (a matrix to E2M1 codes with one E8M0 scale per 32
// values along the contraction, which is its rows or, transposed, its columns) and
// mx4_dequantize (the values that codes stand for).  mxfp6-sm120 page, "Execution
// model" (dynamic quantization with a UE8M0 scale per 32 K values); TokenSpeed SiTU
// page, "Supported contract" (MxE2m1).
//
// A block of 32 values v of the contraction, zeros past its end:
//   rotated   v <- H (signs * v) / sqrt(32), H the 32-point Hadamard matrix: butterflies
//             v[i], v[i + d] <- v[i] + v[i + d], v[i] - v[i + d] at d = 1, 2, 4, 8, 16 in
//             fp32, then one product with the factor.  Two operands rotated alike have
//             the product they had: the rotation only spreads large values over their
//             block.  32 magnitudes below 2^123 add up inside fp32; a block in which larger
//             ones overflow gets the NaN scale.
//   nearest   2^s the scale, s = floor(log2 max|v|) - 2; the code nearest to |v| / 2^s,
//             ties to the even code, at most 6: as mx_quantize does
//   random    s one more where 6 * 2^s < max|v|, so that nothing saturates; with lo <= x
//             <= hi the values next to x = |v| / 2^s, x becomes hi where 256 (x - lo) /
//             (hi - lo) > r + 1/2 for its byte r, i.e. with the probability (x - lo) /
//             (hi - lo), in steps of 1/256: rounding without a bias
// Quotients by 2^s and the differences are exact in fp32, so codes do not depend on
// how they are computed, but for the rotation's own sums, whose order is fixed.
//
// Along rows, a lane takes 8 values and 4 neighbouring lanes a block, so that loads and
// stores of a wave are contiguous; transposed, a workgroup takes 256 rows by 64 columns, a
// thread the 32 rows of one block in two columns (its loads are 128 contiguous bytes of a row
// per 32 lanes), and the codes are regrouped in LDS into 128 contiguous bytes of each output
// row.
//
// Measured (MI355X; bytes at 5 TB/s in brackets): rows 8192 x 7168 bf16 31 us [29], rotated 40 [29]
// (44 where nothing of src is in the last-level cache), at random 49 [41], both 64 [41]; values
// 8192 x 7168 back to bf16 30 [29] (23 where the codes were just written), to fp32 54 [53];
// transposed 16 x 1536 x 4096 fp32 108 [90], 4021 x 2048 bf16 rotated 8 [4], 4021 x 4096 rotated
// and rounded at random 22 [11].  Bound by memory without rotation and random bytes; with them by
// their vector instructions, 11 a value plain, 20 rotated, 35 with both, which are all that a SIMD
// does along rows; transposed (30 a value) they are three quarters of a CU's time, in a launch that
// is one round of workgroups, which load, then compute.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mx_device.h"

namespace moe_mx {

namespace {

constexpr int kThreadsQ = 256;
constexpr float kHadamard = 0.17677669529663687f;  // 1 / sqrt(32)

__device__ __forceinline__ int round_up128(int v) { return (v + 127) & ~127; }

// Shared exponent of a block with largest magnitude amax (fp32 bits); RANDOM: one more from
// 1.5 times a power of two on, 6 * 2^s being 1.5 * 2^(s + 2)
template <bool RANDOM>
__device__ __forceinline__ int exponent4(uint32_t amax) {
  if (!RANDOM) return block_exponent<1>(amax);
  const int E = (int)(amax >> 23);
  return E == 0 ? -127 : max(E - 129 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0), -127);
}

// Code of q = v / 2^s, |q| <= 6, with the complement n of its random byte (r = 255 - n).
// From 1 on, the code's exponent and mantissa bit are the first of the fp32 bits, and those
// behind them, 22 of them, hold (x - lo) / (hi - lo): it is above (r + 1/2) / 256 = (2 r + 1)
// 2^13 / 2^22 where the bits carry once 2^22 - 1 - (2 r + 1) 2^13 = n 2^14 + 2^13 - 1 is added.
// Below 1 codes are 1/2 apart: (1 + x) / 2 has the same bits behind codes 0 and 1, x rounded up
// to 2^-20 first, which passes no multiple of 2^-10 and reaches none from below: being above
// (r + 1/2) / 512 stays as it was.  (13 instructions; with floors and selections 24, and
// 4021 x 4096 rotated, transposed and rounded at random 26 us.)
__device__ __forceinline__ uint32_t random4(float q, uint32_t n) {
  const float x = fabsf(q), small = fmaf(ceilf(x * 0x1p20f), 0x1p-21f, 0.5f);
  const uint32_t bits = __float_as_uint(x < 1.0f ? small : x) + (n << 14) + ((4u << 22) + 8191u);
  // 252 + code, + 4: the code modulo 8, and the sign
  return (bits >> 22 & 7u) | (__float_as_uint(q) >> 28 & 8u);
}

// Scale code of a block; ROTATE: NaN where a rotation has left fp32 (amax infinite or NaN)
template <bool ROTATE>
__device__ __forceinline__ uint8_t scale_code(int s, uint32_t amax) {
  return ROTATE && amax >= 0x7f800000u ? 255 : (uint8_t)(s + 127);
}


// ------------------------------------------------------------- along rows --

struct RowsArgs {
  const void* src;
  int64_t rows;        // of all matrices together
  int64_t ld;
  int cols, units;     // values per row, lanes per row (padded columns / 8)
  const float* signs;
  const uint8_t* random;
  uint8_t* codes;
  uint8_t* scales;
};

constexpr int kUnits = 4;  // pieces of 8 values per thread, a workgroup apart

// VEC: 16-byte pieces of src (and 8 bytes of random) are aligned and lie within a row
// or behind it as a whole
template <bool BF16, bool VEC, bool ROTATE, bool RANDOM>
__global__ __launch_bounds__(kThreadsQ) void k_mx4_rows(RowsArgs a) {
  const int64_t base = (int64_t)blockIdx.x * (kThreadsQ * kUnits);
  const int64_t row0 = base / a.units;
  const uint32_t rem = (uint32_t)(base - row0 * a.units) + threadIdx.x;
  float v[kUnits][8];
  uint32_t rnd[kUnits][2];
  int64_t row[kUnits];
  int col[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t q = rem + kThreadsQ * j, dr = q / (uint32_t)a.units;
    row[j] = row0 + dr;
    col[j] = 8 * (int)(q - dr * (uint32_t)a.units);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    rnd[j][0] = rnd[j][1] = 0;
    if (row[j] >= a.rows) continue;
    const int64_t o = row[j] * a.ld + col[j], ro = row[j] * a.cols + col[j];
    if constexpr (VEC) {
      if (col[j] < a.cols) {
        if constexpr (BF16) {
          const uint4 d = *(const uint4*)((const uint16_t*)a.src + o);
          const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
          const float4* p = (const float4*)((const float*)a.src + o);
          const float4 x = p[0], y = p[1];
          const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = w[i];
        }
        if constexpr (RANDOM) {
          const uint2 d = *(const uint2*)(a.random + ro);
          rnd[j][0] = d.x;
          rnd[j][1] = d.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col[j] + i < a.cols) {
          v[j][i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.src)[o + i] << 16)
                         : ((const float*)a.src)[o + i];
          if constexpr (RANDOM) rnd[j][i / 4] |= (uint32_t)a.random[ro + i] << (8 * (i % 4));
        }
    }
  }
  [[maybe_unused]] float sg[8];
  if constexpr (ROTATE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = a.signs[8 * (threadIdx.x & 3) + i];
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    float(&x)[8] = v[j];
    if constexpr (ROTATE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= sg[i];
#pragma unroll
      for (int d = 1; d < 8; d <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & d)) {
            const float p = x[i], q = x[i + d];
            x[i] = p + q;
            x[i + d] = p - q;
          }
      // distances 8 and 16: the neighbouring lanes
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = lane_move<0xb1>(x[i]);
        x[i] = threadIdx.x & 1 ? o - x[i] : x[i] + o;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = lane_move<0x4e>(x[i]);
        x[i] = (threadIdx.x & 2 ? o - x[i] : x[i] + o) * kHadamard;
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    m = quad_max(m);
    const int s = exponent4<RANDOM>(m);
    const float inv = exp2_neg(s);
    uint32_t w = 0;
    if constexpr (RANDOM) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= random4(x[i] * inv, (~rnd[j][i / 4] >> (8 * (i % 4))) & 255u) << (4 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      w = e2m1_codes(x);
    }
    if (row[j] < a.rows) {
      const int64_t u = row[j] * a.units + (col[j] >> 3);
      *(uint32_t*)(a.codes + 4 * u) = w;
      if ((threadIdx.x & 3) == 0) a.scales[u >> 2] = scale_code<ROTATE>(s, m);
    }
  }
}

// ------------------------------------------------------------- transposed --

struct ColsArgs {
  const void* src;     // [batch, rows, cols], rows ld apart
  int rows, cols;
  int64_t ld;
  int tiles_r, tiles_c;  // of this launch, from column tile first_c on
  int first_c;
  const float* signs;
  const uint8_t* random;  // [batch, rows, cols]
  uint8_t* codes;      // [batch, cols, padded rows / 2]
  uint8_t* scales;
};

constexpr int kTileR = 256, kTileC = 64;

// VEC: two columns of src (and of random) are aligned as a pair
template <bool BF16, bool VEC, bool ROTATE, bool RANDOM>
__global__ __launch_bounds__(kThreadsQ) void k_mx4_cols(ColsArgs a) {
  // a column's 8 blocks of 16 bytes, rows of 9 so that the writes (two columns per
  // lane, a block apart per 32 lanes) spread over the banks
  __shared__ uint4 sc[kTileC][kTileR / 32 + 1];
  __shared__ uint8_t ss[kTileC][kTileR / 32];
  const int tc = a.first_c + blockIdx.x % a.tiles_c, tr = blockIdx.x / a.tiles_c % a.tiles_r;
  const int64_t batch = blockIdx.x / a.tiles_c / a.tiles_r;
  const int pc = threadIdx.x & 31, rb = threadIdx.x >> 5;
  const int c = tc * kTileC + 2 * pc, r0 = tr * kTileR + 32 * rb;
  const int64_t sbase = batch * a.rows * a.ld, rbase = batch * a.rows * a.cols;
  // both columns as they come: bf16 in one word, fp32 in two; two rows' random bytes in one
  uint32_t raw[BF16 ? 1 : 2][32];
  [[maybe_unused]] uint32_t rnd[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) rnd[i] = 0;
  // A tile that lies inside as a whole (the same for all threads) takes its loads without a
  // branch around each, so that all are under way at once.
  auto load = [&](auto inside) {
    constexpr bool IN = decltype(inside)::value;
    const int64_t o0 = sbase + (int64_t)r0 * a.ld + c, ro0 = rbase + (int64_t)r0 * a.cols + c;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      raw[0][i] = 0;
      if constexpr (!BF16) raw[1][i] = 0;
      if (!IN && (r0 + i >= a.rows || c >= a.cols)) continue;
      const int64_t o = o0 + i * a.ld, ro = ro0 + (int64_t)i * a.cols;
      const bool two = IN || VEC || c + 1 < a.cols;
      if constexpr (BF16) {
        const uint16_t* p = (const uint16_t*)a.src + o;
        raw[0][i] = VEC ? *(const uint32_t*)p : p[0] | (two ? (uint32_t)p[1] << 16 : 0u);
      } else {
        const uint32_t* p = (const uint32_t*)a.src + o;
        if constexpr (VEC) {
          const uint2 w = *(const uint2*)p;
          raw[0][i] = w.x;
          raw[1][i] = w.y;
        } else {
          raw[0][i] = p[0];
          if (two) raw[1][i] = p[1];
        }
      }
      if constexpr (RANDOM) {
        const uint8_t* p = a.random + ro;
        const uint32_t w = VEC ? *(const uint16_t*)p : p[0] | (two ? (uint32_t)p[1] << 8 : 0u);
        rnd[i / 2] |= w << (16 * (i % 2));
      }
    }
  };
  if ((tr + 1) * kTileR <= a.rows && (tc + 1) * kTileC <= a.cols) load(std::true_type());
  else load(std::false_type());
  // (one body for both columns: in one round of tiles a CU waits for its code, too; 4021 x 2048
  // bf16 with two bodies 14 us, with one 8)
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if constexpr (BF16) x[i] = __uint_as_float(raw[0][i] << (16 - 16 * h) & 0xffff0000u);
      else x[i] = __uint_as_float(h ? raw[1][i] : raw[0][i]);
    if constexpr (ROTATE) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= a.signs[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(i & d)) {
            const float p = x[i], q = x[i + d];
            x[i] = p + q;
            x[i + d] = p - q;
          }
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= kHadamard;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    const int s = exponent4<RANDOM>(m);
    const float inv = exp2_neg(s);
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[8 * g + i] * inv;
      if constexpr (RANDOM) {
        w[g] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[g] |= random4(y[i], ~rnd[4 * g + i / 2] >> (16 * (i % 2) + 8 * h) & 255u) << (4 * i);
      } else {
        w[g] = e2m1_codes(y);
      }
    }
    sc[2 * pc + h][rb] = make_uint4(w[0], w[1], w[2], w[3]);
    ss[2 * pc + h][rb] = scale_code<ROTATE>(s, m);
  }
  __syncthreads();
  const int padded = round_up128(a.rows);
  const int64_t out0 = batch * a.cols + tc * kTileC;
  const int blocks = (padded - tr * kTileR) >> 5;  // of this tile, 4 or 8 (or more)
#pragma unroll
  for (int i = threadIdx.x; i < kTileC * kTileR / 32; i += kThreadsQ) {
    const int col = i >> 3, b = i & 7;
    if (tc * kTileC + col < a.cols && b < blocks)
      *(uint4*)(a.codes + (out0 + col) * (padded / 2) + (int64_t)tr * (kTileR / 2) + 16 * b) = sc[col][b];
  }
  if (threadIdx.x < 2 * kTileC) {
    const int col = threadIdx.x >> 1, b = 4 * (threadIdx.x & 1);
    if (tc * kTileC + col < a.cols && b < blocks)
      *(uint32_t*)(a.scales + (out0 + col) * (padded / 32) + tr * (kTileR / 32) + b) = *(const uint32_t*)&ss[col][b];
  }
}

// ----------------------------------------------------------------- values --

typedef float v2f __attribute__((ext_vector_type(2)));

// 8 values per thread and step.  VEC: 16-byte pieces of dst are aligned.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreadsQ) void k_mx4_values(const uint32_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int64_t total,
                                                          int units, void* __restrict__ dst, int64_t ld) {
  for (int64_t u = (int64_t)blockIdx.x * kThreadsQ + threadIdx.x; u < total; u += (int64_t)gridDim.x * kThreadsQ) {
    const uint32_t w = codes[u], e = scales[u >> 2];
    const float s = e == 255 ? __builtin_nanf("") : e8m0_to_f32(e);
    const v2f p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const v2f p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const v2f p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const float x[8] = {p0[0] * s, p0[1] * s, p1[0] * s, p1[1] * s, p2[0] * s, p2[1] * s, p3[0] * s, p3[1] * s};
    int64_t o = 8 * u;
    if (ld != 8 * (int64_t)units) {  // (uniform: a division per piece only where rows are apart)
      const int64_t row = u / units;
      o = row * ld + 8 * (u - row * units);
    }
    if constexpr (BF16) {
      // exact: two bits of mantissa, and bf16 has fp32's exponents (below 2^-126 too:
      // multiples of 2^-128)
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
      uint16_t* p = (uint16_t*)dst + o;
      if constexpr (VEC) {
        *(uint4*)p = make_uint4(h[0], h[1], h[2], h[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
      }
    } else {
      float* p = (float*)dst + o;
      if constexpr (VEC) {
        ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i];
      }
    }
  }
}

// ----------------------------------------------------- E4M3 codes of E2M1 --

// E4M3 codes of the eight E2M1 codes of a word: every E2M1 value is an E4M3 value.
__device__ __forceinline__ uint2 e4m3_of_e2m1(uint32_t w) {
  constexpr uint32_t lo = 0x3c383000u, hi = 0x4c484440u;  // codes of 0, .5, 1, 1.5 and of 2, 3, 4, 6
  const uint32_t a = w & 0x0f0f0f0fu, b = (w >> 4) & 0x0f0f0f0fu;
  const uint32_t even = __builtin_amdgcn_perm(hi, lo, a & 0x07070707u) | (a & 0x08080808u) << 4;
  const uint32_t odd = __builtin_amdgcn_perm(hi, lo, b & 0x07070707u) | (b & 0x08080808u) << 4;
  return make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u), __builtin_amdgcn_perm(odd, even, 0x07030602u));
}

__global__ __launch_bounds__(kThreadsQ) void k_mx4_expand(const uint32_t* __restrict__ codes, int64_t words,
                                                          uint2* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * kThreadsQ + threadIdx.x; i < words; i += (int64_t)gridDim.x * kThreadsQ)
    out[i] = e4m3_of_e2m1(codes[i]);
}

// ------------------------------------------------------------------- host --

constexpr int64_t kMaxDim = (int64_t)1 << 30;  // rows, columns, matrices
// Workgroups of one launch, which has fewer than 2^32 threads; what has more takes several.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;

// F with the four choices as compile-time constants
template <class F>
void for_choices(bool bf16, bool vec, bool rotate, bool random, F f) {
  auto last = [&](auto A, auto B, auto C) {
    if (random) f(A, B, C, std::true_type());
    else f(A, B, C, std::false_type());
  };
  auto third = [&](auto A, auto B) {
    if (rotate) last(A, B, std::true_type());
    else last(A, B, std::false_type());
  };
  auto second = [&](auto A) {
    if (vec) third(A, std::true_type());
    else third(A, std::false_type());
  };
  if (bf16) second(std::true_type());
  else second(std::false_type());
}

}  // namespace

hipError_t launch_mx4_expand(const uint8_t* codes, int64_t bytes, uint8_t* out, hipStream_t stream) {
  const int64_t words = bytes / 4;
  if (words == 0) return hipSuccess;
  const unsigned blocks = (unsigned)std::min<int64_t>((words + kThreadsQ - 1) / kThreadsQ, 1 << 16);
  k_mx4_expand<<<blocks, kThreadsQ, 0, stream>>>((const uint32_t*)codes, words, (uint2*)out);
  return hipGetLastError();
}

}  // namespace moe_mx

using namespace moe_mx;

extern "C" moe_status_t mx4_quantize(const void* src, moe_src_t src_dtype, int64_t batch, int64_t rows, int64_t cols,
                                     int64_t src_ld, int transpose, const float* signs, const uint8_t* random,
                                     uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if ((src_dtype != MOE_SRC_BF16 && src_dtype != MOE_SRC_FP32) || batch < 0 || rows < 0 || cols < 1 || src_ld < cols ||
      (transpose != 0 && transpose != 1))
    return MOE_ERR_INVALID_ARG;
  if (rows > kMaxDim || cols > kMaxDim || batch > kMaxDim || (double)batch * rows * src_ld > 1.4e14)
    return MOE_ERR_UNSUPPORTED;
  const bool bf16 = src_dtype == MOE_SRC_BF16;
  const int64_t es = bf16 ? 2 : 4;
  if (batch == 0 || rows == 0) return MOE_OK;
  if (!src || !codes || !scales || !aligned(src, es) || !aligned(codes, 16) || !aligned(scales, 4) ||
      !aligned(signs, 4))
    return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  if (transpose) {
    const int64_t tiles_r = (rows + kTileR - 1) / kTileR, tiles_c = (cols + kTileC - 1) / kTileC;
    // matrices of a launch and column tiles (tiles_r <= 2^22)
    const int64_t nb = std::max<int64_t>(kMaxBlocks / (tiles_r * tiles_c), 1), nc = std::min(tiles_c, kMaxBlocks / tiles_r);
    const int64_t padded = (rows + 127) / 128 * 128;
    const bool vec = cols % 2 == 0 && src_ld % 2 == 0 && aligned(src, 2 * es) && (!random || aligned(random, 2));
    for (int64_t b = 0; b < batch; b += nb)
      for (int64_t c = 0; c < tiles_c; c += nc) {
        const int64_t n = std::min(nc, tiles_c - c);
        ColsArgs a = {(const char*)src + b * rows * src_ld * es, (int)rows, (int)cols, src_ld, (int)tiles_r, (int)n, (int)c,
                      signs, random ? random + b * rows * cols : nullptr, codes + b * cols * (padded / 2),
                      scales + b * cols * (padded / 32)};
        const int64_t blocks = std::min(nb, batch - b) * tiles_r * n;
        for_choices(bf16, vec, signs != nullptr, random != nullptr, [&](auto B, auto V, auto R, auto S) {
          k_mx4_cols<B.value, V.value, R.value, S.value><<<(unsigned)blocks, kThreadsQ, 0, stream>>>(a);
        });
        if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
      }
  } else {
    const int64_t all = batch * rows, units = (cols + 127) / 128 * 16, nr = kMaxBlocks * (kThreadsQ * kUnits) / units;
    const bool vec = cols % 8 == 0 && src_ld * es % 16 == 0 && aligned(src, 16) &&
                     (!random || aligned(random, 8));
    for (int64_t r = 0; r < all; r += nr) {
      RowsArgs a = {(const char*)src + r * src_ld * es, std::min(nr, all - r), src_ld, (int)cols, (int)units, signs,
                    random ? random + r * cols : nullptr, codes + 4 * r * units, scales + r * units / 4};
      const int64_t blocks = (a.rows * units + kThreadsQ * kUnits - 1) / (kThreadsQ * kUnits);
      for_choices(bf16, vec, signs != nullptr, random != nullptr, [&](auto B, auto V, auto R, auto S) {
        k_mx4_rows<B.value, V.value, R.value, S.value><<<(unsigned)blocks, kThreadsQ, 0, stream>>>(a);
      });
      if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
    }
  }
  return MOE_OK;
}

extern "C" moe_status_t mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                       void* dst, moe_src_t dst_dtype, int64_t dst_ld, hipStream_t stream) {
  if ((dst_dtype != MOE_SRC_BF16 && dst_dtype != MOE_SRC_FP32) || rows < 0 || cols < 1 || cols % 32 || dst_ld < cols)
    return MOE_ERR_INVALID_ARG;
  if (rows > kMaxDim || cols > kMaxDim || (double)rows * dst_ld > 1.4e14) return MOE_ERR_UNSUPPORTED;
  const bool bf16 = dst_dtype == MOE_SRC_BF16;
  const int64_t es = bf16 ? 2 : 4;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !dst || !aligned(codes, 4) || !aligned(dst, es)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  const bool vec = dst_ld * es % 16 == 0 && aligned(dst, 16);
  const int64_t total = rows * (cols / 8);
  const unsigned blocks = (unsigned)std::min<int64_t>((total + kThreadsQ - 1) / kThreadsQ, 1 << 16);
#define MX4_VALUES(B, V)                                                                                          \
  k_mx4_values<B, V><<<blocks, kThreadsQ, 0, stream>>>((const uint32_t*)codes, scales, total, (int)(cols / 8), dst, \
                                                       dst_ld)
  if (bf16 && vec) MX4_VALUES(true, true);
  else if (bf16) MX4_VALUES(true, false);
  else if (vec) MX4_VALUES(false, true);
  else MX4_VALUES(false, false);
#undef MX4_VALUES
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
