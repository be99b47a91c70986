// mx_linear for a handful of rows: 16-row tiles, the contraction split over the
// waves of a workgroup.
//
// One token's projection is bound by latency before bandwidth (15.6 MB of weights
// through 4096 x 7168 are 3 us of HBM): the weights have to be spread over the
// whole chip and requested at once, in one launch.  So a workgroup takes 16
// columns of one tile and its 8 waves take turns along K (two 128-K chunks each,
// side by side, so that a row's reads stay in 128-byte lines), each with kAhead
// chunks in flight in registers; the partial sums meet in LDS, are added in wave
// order (deterministic) and finished by the epilogue, whose operands were requested
// before the first chunk.  Weights go straight from memory to the MFMA's first
// operand, activations to the second; rows past the tile load nothing.  Every lane
// then reads another row, which costs the cache lookups that the LDS copies of
// gemm_rows.hip save: from about 16 rows on those win in spite of a second launch.
// (One token, 4096 x 7168 E2M1 x bf16: 8.0 us a call against 11.6 for 16-row LDS
// tiles in 7 K ranges and their join; 16 rows 12.9 against 12.1.)
//
// Lane layouts are those of the stream kernels (gemm_stream.hip).  QUANT: bf16 rows
// are quantized to MXFP8 on the way, the same codes and scales as mx_quantize: lane
// g of a row holds values [16g, +16) and [64 + 16g, +16) of a chunk, i.e. halves of
// blocks g/2 and 2 + g/2, so a block's largest magnitude is one exchange away;
// the MFMA takes from lane g the scale of block g.  (A launch to quantize costs
// 2.5 us.)
#include <hip/hip_runtime.h>

#include "epilogue.h"
#include "gemm.h"
#include "mx_device.h"

namespace moe_mx {

namespace {

typedef int v6i __attribute__((ext_vector_type(6)));
typedef __bf16 v32bf __attribute__((ext_vector_type(32)));
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));

constexpr int kAhead = 4;  // chunks in flight per wave
constexpr int W = 8;       // waves

// activations: bf16 as given, E4M3 codes with scales, bf16 quantized here
enum Act { kBf16 = 0, kMx = 1, kQuant = 2 };

struct Chunk {
  uint4 a[4];         // kBf16: 32 values; kQuant: 2 x 16 values; kMx: a[0], a[1] codes
  uint32_t as;        // kMx: the chunk's four scale bytes
  uint32_t b[6];      // weights; E2M1: 4 dwords, E3M2: 6
  uint32_t bs;        // the chunk's four scale bytes
};

template <int ACT, int WF>
__device__ __forceinline__ void load_chunk(Chunk& f, const uint8_t* arow, const uint8_t* asrow, const uint8_t* brow,
                                           const uint8_t* bsrow, int c, int g) {
  if (WF == 1) {
    const uint4 v = *(const uint4*)(brow + 64 * (int64_t)c + 16 * g);
    f.b[0] = v.x; f.b[1] = v.y; f.b[2] = v.z; f.b[3] = v.w;
  } else {
    // 24 bytes on an 8-byte address
    const uint8_t* q = brow + 24 * (4 * (int64_t)c + g);
    const u32x4_a8 x = *(const u32x4_a8*)q;
    const uint2 y = *(const uint2*)(q + 16);
    f.b[0] = x[0]; f.b[1] = x[1]; f.b[2] = x[2]; f.b[3] = x[3]; f.b[4] = y.x; f.b[5] = y.y;
  }
  f.bs = *(const uint32_t*)(bsrow + 4 * c);
  if (arow == nullptr) return;  // a row past the tile: zeros, set once
  if (ACT == kBf16) {
    const uint4* q = (const uint4*)(arow + 2 * (128 * (int64_t)c + 32 * g));
#pragma unroll
    for (int i = 0; i < 4; ++i) f.a[i] = q[i];
  } else if (ACT == kQuant) {
    const uint4* q = (const uint4*)(arow + 2 * (128 * (int64_t)c + 16 * g));
    f.a[0] = q[0]; f.a[1] = q[1];
    f.a[2] = q[8]; f.a[3] = q[9];
  } else {
    f.a[0] = *(const uint4*)(arow + 128 * (int64_t)c + 16 * g);
    f.a[1] = *(const uint4*)(arow + 128 * (int64_t)c + 64 + 16 * g);
    f.as = *(const uint32_t*)(asrow + 4 * c);
  }
}

// 16 bf16 values (two uint4) to 16 E4M3 codes, divided by 2^s
__device__ __forceinline__ uint4 quant16(const uint4& lo, const uint4& hi, float inv) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = e4m3_pair(__uint_as_float(w[2 * q] << 16) * inv, __uint_as_float(w[2 * q] & 0xffff0000u) * inv) |
           (e4m3_pair(__uint_as_float(w[2 * q + 1] << 16) * inv, __uint_as_float(w[2 * q + 1] & 0xffff0000u) * inv)
            << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// largest magnitude (fp32 bits) of 16 bf16 values
__device__ __forceinline__ uint32_t amax16(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, max((w[q] << 16) & 0x7fffffffu, w[q] & 0x7fff0000u));
  return m;
}

template <int ACT, int WF>
__device__ __forceinline__ void mul_chunk(v4f& acc, const Chunk& f, int g, int r) {
  const int wsc = (int)((f.bs >> (8 * g)) & 0xffu);
  if (ACT == kBf16) {
    const float sc = e8m0_to_f32(wsc);
    v32bf wide;
    if (WF == 2)
      wide = __builtin_amdgcn_cvt_scalef32_pk32_bf16_bf6(
          (v6i){(int)f.b[0], (int)f.b[1], (int)f.b[2], (int)f.b[3], (int)f.b[4], (int)f.b[5]}, sc);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8bf bv;
      if (WF == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) bv[i] = wide[8 * s + i];
      } else {
        const v2bf q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.b[s], sc, 0);
        const v2bf q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.b[s], sc, 1);
        const v2bf q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.b[s], sc, 2);
        const v2bf q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.b[s], sc, 3);
        bv = (v8bf){q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
      }
      v8bf av;
      __builtin_memcpy(&av, &f.a[s], 16);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, av, acc, 0, 0, 0);
    }
    return;
  }
  uint4 lo = f.a[0], hi = f.a[1];
  int asc;
  if (ACT == kQuant) {
    uint32_t m1 = amax16(f.a[0], f.a[1]), m2 = amax16(f.a[2], f.a[3]);
    m1 = max(m1, (uint32_t)__shfl_xor((int)m1, 16));
    m2 = max(m2, (uint32_t)__shfl_xor((int)m2, 16));
    const int s1 = block_exponent<3>(m1), s2 = block_exponent<3>(m2);
    lo = quant16(f.a[0], f.a[1], exp2_neg(s1));
    hi = quant16(f.a[2], f.a[3], exp2_neg(s2));
    // blocks 0, 1 are the first of lanes g = 0, 2; blocks 2, 3 their second
    const int src = 32 * (g & 1) + r;
    const int t1 = __shfl(s1, src), t2 = __shfl(s2, src);
    asc = (g >> 1 ? t2 : t1) + 127;
  } else {
    asc = (int)((f.as >> (8 * g)) & 0xffu);
  }
  const v8i av = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  const v8i bv = {(int)f.b[0], (int)f.b[1], (int)f.b[2], (int)f.b[3],
                  WF == 2 ? (int)f.b[4] : 0, WF == 2 ? (int)f.b[5] : 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc, Fmt<WF>::MFMA, 0, 0, wsc, 0, asc);
}

// Tile ti of the list that k_group_tiles would make (16 rows each, groups in order,
// ends clamped so that they ascend within [0, M]), by each wave on its own: a lane
// takes a run of groups.  rows = 0 behind the last tile.  (A launch that writes the
// list costs a call of a few rows more than its product: 4 rows over 11 groups, 232
// x 512, 4.7 us a call against 8.3.)
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int groups, int M, int ti) {
  const int lane = threadIdx.x & 63, per = (groups + 63) >> 6, g0 = lane * per, g1 = min(g0 + per, groups);
  const int64_t first = offsets[0];
  auto end = [&](int g) { return (int32_t)min(max((int64_t)offsets[g + 1] - first, (int64_t)0), (int64_t)M); };
  int32_t last = 0;
  for (int g = g0; g < g1; ++g) last = max(last, end(g));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t v = __shfl_up(last, d);
    if (lane >= d) last = max(last, v);
  }
  int32_t start = __shfl_up(last, 1);
  if (lane == 0) start = 0;
  int32_t s = start, n = 0;
  for (int g = g0; g < g1; ++g) {
    const int32_t e = max(s, end(g));
    n += (e - s + 15) >> 4;
    s = e;
  }
  int32_t upto = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  Tile t = {0, 0, 0, 0};
  int c = ti - (upto - n);  // the tile's place in this lane's run
  const uint64_t holder = __ballot(c >= 0 && c < n);
  if (holder == 0) return t;
  s = start;
  for (int g = g0; g < g1; ++g) {
    const int32_t e = max(s, end(g)), nt = (e - s + 15) >> 4;
    if (c >= 0 && c < nt) t = {g, s + 16 * c, min(16, e - s - 16 * c), 0};
    c -= nt;
    s = e;
  }
  const int src = __builtin_ctzll(holder);
  t.expert = __builtin_amdgcn_readlane(t.expert, src);
  t.p0 = __builtin_amdgcn_readlane(t.p0, src);
  t.rows = __builtin_amdgcn_readlane(t.rows, src);
  return t;
}

template <int ACT, int WF>
__global__ __launch_bounds__(64 * W) void k_linear_few(FcArgs p) {
  __shared__ float part[W][16][kFewCols + 4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const int nch = blockIdx.x % p.nchunks, ti = blockIdx.x / p.nchunks;
  const int N = p.N, K = p.K, col0 = nch * kFewCols;
  Tile t;
  if (p.dense_rows > 0) {
    t.expert = 0;
    t.p0 = 16 * ti;
    t.rows = min(16, p.dense_rows - 16 * ti);
  } else {
    t = find_tile(p.group_offsets, p.groups, p.group_rows, ti);
    if (t.rows == 0) return;
  }
  // the first 32 threads finish a piece of out each
  const int prow = threadIdx.x >> 1, pcol = col0 + 8 * (threadIdx.x & 1);
  const bool piece = threadIdx.x < 32 && prow < t.rows && pcol < N;
  const int64_t o = (int64_t)(t.p0 + prow) * N + pcol;
  EpiIn in = {};
  EpiBias bias = {};
  if (piece) {
    in = epi_in(p.epi, o);
    bias = epi_bias(p.epi, N, t.expert, pcol);
  }

  const uint8_t* arow = nullptr;
  const uint8_t* asrow = nullptr;
  if (r < t.rows) {
    const int64_t row = t.p0 + r;
    arow = (const uint8_t*)p.a + row * (ACT == kMx ? K : 2 * (int64_t)K);
    if (ACT == kMx) asrow = p.a_scale + row * (K / 32);
  }
  // columns past N read the last weight row and are not stored
  const int64_t wrow = min(col0 + r, N - 1);
  const uint8_t* brow = p.w + (int64_t)t.expert * p.w_estride + wrow * ((int64_t)K * Fmt<WF>::BITS / 8);
  const uint8_t* bsrow = p.w_scale + (int64_t)t.expert * p.ws_estride + wrow * (K / 32);
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  Chunk f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    f[u].as = 0x7f7f7f7fu;
#pragma unroll
    for (int q = 0; q < 4; ++q) f[u].a[q] = make_uint4(0, 0, 0, 0);
  }
  // the wave's chunks: pairs w, w + W, ... of neighbouring chunks
  const int nchunk = K / 128;
  auto chunk = [&](int i) { return 2 * (w + W * (i >> 1)) + (i & 1); };
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (chunk(u) < nchunk) load_chunk<ACT, WF>(f[u], arow, asrow, brow, bsrow, chunk(u), g);
  for (int i = 0; chunk(i) < nchunk; i += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (chunk(i + u) < nchunk) mul_chunk<ACT, WF>(acc, f[u], g, r);
      if (chunk(i + u + kAhead) < nchunk) load_chunk<ACT, WF>(f[u], arow, asrow, brow, bsrow, chunk(i + u + kAhead), g);
    }
  }
  // weights first: the lane holds row r, columns 4g .. 4g + 3
  *(float4*)&part[w][r][4 * g] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (!piece) return;
  float v[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) v[h] = epi_bias_at(p.epi, bias, h);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float* s = &part[i][prow][pcol - col0];
    const float4 lo = *(const float4*)s, hi = *(const float4*)(s + 4);
    const float a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int h = 0; h < 8; ++h) v[h] += a[h];
  }
  epi_store(p.epi, o, in, v);
}

template <int ACT, int WF>
void launch_few_t(const FcArgs& p, int ntiles, hipStream_t st) {
  k_linear_few<ACT, WF><<<(unsigned)((int64_t)ntiles * p.nchunks), 64 * W, 0, st>>>(p);
}

}  // namespace

hipError_t launch_linear_few(const FcArgs& p, bool mx_act, bool quant, int wfmt, hipStream_t st) {
  const int ntiles = p.dense_rows > 0 ? (p.dense_rows + 15) / 16 : p.max_tiles;
  if (ntiles == 0) return hipSuccess;
  if (quant) {
    if (wfmt == 1) launch_few_t<kQuant, 1>(p, ntiles, st);
    else launch_few_t<kQuant, 2>(p, ntiles, st);
  } else if (mx_act) {
    if (wfmt == 1) launch_few_t<kMx, 1>(p, ntiles, st);
    else launch_few_t<kMx, 2>(p, ntiles, st);
  } else {
    if (wfmt == 1) launch_few_t<kBf16, 1>(p, ntiles, st);
    else launch_few_t<kBf16, 2>(p, ntiles, st);
  }
  return hipGetLastError();
}

}  // namespace moe_mx
