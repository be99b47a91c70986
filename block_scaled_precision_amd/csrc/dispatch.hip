// Dispatch of a batch's rows to the experts and back, as operators of their
// own: moe_permute, moe_unpermute, their gradients and the router's gradient
// (mxfp6-sm120 page, "Execution model": indirect routing and the unpermuting
// reduction; TokenSpeed SiTU page, "Supported contract": expert shards).
//
// With row p = row_of[t, j] of assignment (t, j), -1 where there is none:
//   permute            rows[p] = x[t]
//   its gradient       dx[t] = sum_j drows[p]
//   unpermute          y[t] = residual[t] + sum_j w[t, j] rows[p]
//   its gradient       drows[p] = w[t, j] dy[t],  dw[t, j] = <dy[t], rows[p]>
// The gradient of permute is unpermute without weights or residual.  Sums are
// held in fp32 and added in slot order, and each output is rounded once; no
// order depends on scheduling, so results repeat bit for bit.
//
// All of them move rows and compute next to nothing: the bound is memory
// traffic (or, for a few tokens, the launch).  Work is therefore laid out so
// that each row is read once and written once: the gathers and the sums hold
// one 16-byte piece of a token's row per thread and walk its k rows with up to
// kSlots of them in flight.  Rows whose address or stride is not a multiple of
// 16 bytes, or whose length is not a whole number of 16-byte pieces, go
// element by element.
#include <hip/hip_runtime.h>

#include "internal.h"

namespace moe_mx {

namespace {

constexpr int kSlots = 8;            // rows of a token in flight per thread
constexpr int64_t kMaxBlocks = 1 << 20;
constexpr int kThreadsD = 256;

// Row elements: V of type T per access.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
  T v[V];
};
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Threads of a workgroup are groups of `tpr` neighbours, one row per group;
// thread c of a group owns piece c of the row's column block.
struct RowMap {
  int tpr, lg;       // threads per row (a power of two) and its logarithm
  int pieces;        // pieces per row
  int cblocks;       // column blocks of tpr pieces
  int64_t nrows;     // rows
  int64_t nblocks;   // workgroup-sized units of work
};

// The widest group of at most 256 threads that leaves at most an eighth of its
// threads without a piece; rows shorter than 64 pieces take the next power of
// two, so that short rows share a wave.
RowMap row_map(int64_t nrows, int64_t pieces) {
  RowMap m;
  int lg = 8;
  if (pieces < 64) {
    lg = 0;
    while ((1 << lg) < pieces) ++lg;
  } else {
    for (; lg > 6; --lg) {
      const int64_t t = (int64_t)1 << lg, span = (pieces + t - 1) / t * t;
      if ((span - pieces) * 8 <= span) break;
    }
  }
  m.lg = lg;
  m.tpr = 1 << lg;
  m.pieces = (int)pieces;
  m.cblocks = (int)((pieces + m.tpr - 1) / m.tpr);
  m.nrows = nrows;
  const int64_t rpb = kThreadsD >> lg;
  m.nblocks = (nrows + rpb - 1) / rpb * m.cblocks;
  return m;
}

// The same with U pieces per thread, tpr apart.
RowMap with_pieces(RowMap m, int U) {
  m.nblocks = m.nblocks / m.cblocks * ((m.cblocks + U - 1) / U);
  m.cblocks = (m.cblocks + U - 1) / U;
  return m;
}

// (row, first piece) of this thread in unit b, or false
template <int U = 1>
__device__ __forceinline__ bool row_piece(const RowMap& m, int64_t b, int64_t& row, int& c) {
  const int64_t rb = b / m.cblocks;
  const int cb = (int)(b - rb * m.cblocks);
  row = rb * (kThreadsD >> m.lg) + (threadIdx.x >> m.lg);
  c = cb * m.tpr * U + (threadIdx.x & (m.tpr - 1));
  return row < m.nrows && c < m.pieces;
}

unsigned grid_blocks(int64_t n) { return (unsigned)(n < 1 ? 1 : n > kMaxBlocks ? kMaxBlocks : n); }

// Local segment [base, end) of sorted_assign, within its A entries
__device__ __forceinline__ void local_segment(const int32_t* offsets, int lo, int n, int64_t A, int64_t& base,
                                              int64_t& end) {
  base = min((int64_t)max(offsets[lo], 0), A);
  end = max(min((int64_t)max(offsets[lo + n], 0), A), base);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16-byte accesses to a matrix too large to stay in the caches (STREAM) bypass
// their retention
template <bool STREAM, typename P>
__device__ __forceinline__ P load_piece(const P* p) {
  if constexpr (STREAM && sizeof(P) == 16) {
    const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);
    P r;
    __builtin_memcpy(&r, &v, 16);
    return r;
  } else {
    return *p;
  }
}
template <bool STREAM, typename P>
__device__ __forceinline__ void store_piece(P* p, const P& v) {
  if constexpr (STREAM && sizeof(P) == 16) {
    u32x4 r;
    __builtin_memcpy(&r, &v, 16);
    __builtin_nontemporal_store(r, (u32x4*)p);
  } else {
    *p = v;
  }
}
// Outputs from this size on are stored past the caches, and the rows of
// moe_unpermute_backward, whose rows and drows then exceed them several times
// over, are loaded past them too.  (With a piece per thread: gradient of 4096 x 4096
// fp32 tokens 52 us against 55; 2047 x 5120 bf16 tokens, half of their rows local, 22.4
// against 34, as the rows stay in the last-level cache; gradient of 8192 x 4096 bf16
// tokens 226 against 239.  Outputs of decode batches stay cached for their reader.)
constexpr int64_t kStreamBytes = 16 << 20;

// ------------------------------------------------------------- permute ---

// Rows of at least this many bytes in all: a launch that inverts sorted_assign,
// then one that reads each token's row once for all of its rows.  Below it one
// launch gathers row by row, reading x up to k times, from the caches.  (bf16, H
// 7168, k 8: 8192 tokens 219 us against 364, 1024 tokens 31.8 against 35.9, 256
// tokens 11.5 against 10.3, one token 11.9 against 8.7; in elements, H 4095, k 8: 4096
// tokens 110 against 133.)
constexpr int64_t kTokenBytes = 64 << 20;
// Rows that only elements of 2 or 4 bytes can walk (odd lengths, strides or
// addresses): workgroups of a piece per thread from which on each takes four.
constexpr int64_t kElementBlocks = 8192;

// row_of[a] of every assignment a
__global__ __launch_bounds__(kThreadsD) void k_invert(int64_t A, const int32_t* __restrict__ offsets,
                                                      const int32_t* __restrict__ sorted_assign, int lo, int n,
                                                      int64_t num_rows, int32_t* __restrict__ row_of) {
  int64_t base, end;
  local_segment(offsets, lo, n, A, base, end);
  for (int64_t g = (int64_t)blockIdx.x * kThreadsD + threadIdx.x; g < A; g += (int64_t)gridDim.x * kThreadsD) {
    const int32_t a = sorted_assign[g];
    if (a >= 0 && a < A) row_of[a] = g >= base && g < end && g - base < num_rows ? (int32_t)(g - base) : -1;
  }
}

// One row per token: each piece is read once and written to the token's rows.
template <typename P>
__global__ __launch_bounds__(kThreadsD) void k_permute_tokens(RowMap m, const P* __restrict__ x, int64_t x_ld, int k,
                                                              const int32_t* __restrict__ row_of,
                                                              P* __restrict__ rows, int64_t rows_ld,
                                                              int64_t num_rows) {
  for (int64_t b = blockIdx.x; b < m.nblocks; b += gridDim.x) {
    int64_t t;
    int c;
    if (!row_piece(m, b, t, c)) continue;
    const P v = x[t * x_ld + c];
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      int32_t p[kSlots];
#pragma unroll
      for (int q = 0; q < kSlots; ++q) p[q] = j0 + q < k ? row_of[t * k + j0 + q] : -1;
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (p[q] >= 0 && p[q] < num_rows) rows[(int64_t)p[q] * rows_ld + c] = v;
    }
  }
}

// One row per assignment g of sorted_assign: row g - base is the row of its
// token; thread 0 of the row notes where it went.  U pieces per thread.
template <typename P, int U>
__global__ __launch_bounds__(kThreadsD) void k_permute_rows(RowMap m, const P* __restrict__ x, int64_t x_ld, int k,
                                                            const int32_t* __restrict__ offsets,
                                                            const int32_t* __restrict__ sorted_assign, int lo, int n,
                                                            P* __restrict__ rows, int64_t rows_ld, int64_t num_rows,
                                                            int32_t* __restrict__ row_of) {
  int64_t base, end;
  local_segment(offsets, lo, n, m.nrows, base, end);
  for (int64_t b = blockIdx.x; b < m.nblocks; b += gridDim.x) {
    int64_t g;
    int c;
    if (!row_piece<U>(m, b, g, c)) continue;
    const int32_t a = sorted_assign[g];
    if (a < 0 || a >= m.nrows) continue;
    const bool here = g >= base && g < end && g - base < num_rows;
    if (c == 0) row_of[a] = here ? (int32_t)(g - base) : -1;
    if (!here) continue;
    P v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = x[(int64_t)(a / k) * x_ld + min(c + u * m.tpr, m.pieces - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * m.tpr < m.pieces) rows[(g - base) * rows_ld + c + u * m.tpr] = v[u];
  }
}

// ----------------------------------------------------------- unpermute ---

// y[t] = residual[t] + sum over slots j of (w[t, j]) rows[row_of[t, j]]; U pieces,
// tpr apart, per thread.  A thread waits for row_of and then for the rows; in large
// calls several pieces per wait keep more of them in flight (gradients of permute:
// 4096 x 4096 fp32 tokens with a quarter of their rows 43 against 55 us, bf16 17.5
// against 40; 8192 x 7168 bf16 198 against 247; 4096 x 4095 bf16 in elements 74
// against 175).  Four pieces of 16 bytes take too many registers (8192 x 7168 with
// weights 463 us against 255).
template <typename T, int V, bool WEIGHTED, bool STREAM, int U>
__global__ __launch_bounds__(kThreadsD) void k_gather_sum(RowMap m, const T* __restrict__ rows, int64_t rows_ld,
                                                          int num_rows, const int32_t* __restrict__ row_of,
                                                          const float* __restrict__ w, int k, const T* residual,
                                                          int64_t res_ld, T* y, int64_t y_ld) {
  using P = Pack<T, V>;
  for (int64_t b = blockIdx.x; b < m.nblocks; b += gridDim.x) {
    int64_t t;
    int c0;
    if (!row_piece<U>(m, b, t, c0)) continue;
    int64_t c[U];  // past the row: its last piece again, not stored
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = (int64_t)min(c0 + u * m.tpr, m.pieces - 1) * V;
    float s[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (residual) {
        const P r = *(const P*)(residual + t * res_ld + c[u]);
#pragma unroll
        for (int q = 0; q < V; ++q) s[u][q] = to_f32(r.v[q]);
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) s[u][q] = 0.f;
      }
    }
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      P v[kSlots][U];
      float wt[kSlots];
      bool use[kSlots];
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        const int32_t p = j0 + q < k ? row_of[t * k + j0 + q] : -1;
        use[q] = p >= 0 && p < num_rows;
        wt[q] = WEIGHTED && use[q] ? w[t * k + j0 + q] : 1.f;
        if (use[q]) {
#pragma unroll
          for (int u = 0; u < U; ++u) v[q][u] = *((const P*)(rows + (int64_t)p * rows_ld + c[u]));
        }
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (use[q]) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i)
              s[u][i] = WEIGHTED ? fmaf(wt[q], to_f32(v[q][u].v[i]), s[u][i]) : s[u][i] + to_f32(v[q][u].v[i]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      P o;
#pragma unroll
      for (int q = 0; q < V; ++q) o.v[q] = (T)s[u][q];
      if (c0 + u * m.tpr < m.pieces) store_piece<STREAM>((P*)(y + t * y_ld + c[u]), o);
    }
  }
}

// drows[row_of[t, j]] = w[t, j] dy[t] and dw[t, j] = <dy[t], rows[row_of[t, j]]>:
// one workgroup of TH threads per Q slots of a token, each thread holding one
// partial dot product per slot over its pieces of the row.
template <typename T, int V, bool STREAM, int TH, int Q>
__global__ __launch_bounds__(TH) void k_unpermute_grad(int64_t tokens, int pieces, const T* __restrict__ dy,
                                                       int64_t dy_ld, const T* __restrict__ rows, int64_t rows_ld,
                                                       int num_rows, const int32_t* __restrict__ row_of,
                                                       const float* __restrict__ w, int k, T* __restrict__ drows,
                                                       int64_t drows_ld, float* __restrict__ dw) {
  using P = Pack<T, V>;
  __shared__ float part[TH / 64][Q];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, parts = (k + Q - 1) / Q;
  for (int64_t i = blockIdx.x; i < tokens * parts; i += gridDim.x) {
    const int64_t t = i / parts;
    const int j0 = Q * (int)(i % parts);
    int32_t p[Q];
    float wt[Q], dot[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      p[q] = j0 + q < k ? row_of[t * k + j0 + q] : -1;
      if (p[q] >= num_rows) p[q] = -1;
      wt[q] = p[q] >= 0 ? w[t * k + j0 + q] : 0.f;
      dot[q] = 0.f;
    }
    for (int c = threadIdx.x; c < pieces; c += TH) {
      const P g = *(const P*)(dy + t * dy_ld + (int64_t)c * V);
      P v[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (p[q] >= 0) v[q] = load_piece<STREAM>((const P*)(rows + (int64_t)p[q] * rows_ld + (int64_t)c * V));
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (p[q] >= 0) {
          P o;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float ge = to_f32(g.v[e]);
            dot[q] = fmaf(ge, to_f32(v[q].v[e]), dot[q]);
            o.v[e] = (T)(wt[q] * ge);
          }
          store_piece<STREAM>((P*)(drows + (int64_t)p[q] * drows_ld + (int64_t)c * V), o);
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) dot[q] += __shfl_xor(dot[q], d);
      if (lane == 0) part[wv][q] = dot[q];
    }
    __syncthreads();
    if (threadIdx.x < Q && j0 + (int)threadIdx.x < k) {
      float s = part[0][threadIdx.x];
#pragma unroll
      for (int u = 1; u < TH / 64; ++u) s += part[u][threadIdx.x];
      dw[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// -------------------------------------------------------- router gradient ---

// The weights of a token are the softmax of its chosen logits, so
//   dlogits[t, e_j] = w_j (dw_j - sum_i w_i dw_i), and 0 for the others.
// One wave per token builds the row in LDS (zeros, then the chosen entries) and
// writes it out with neighbouring lanes on neighbouring columns.  Ids outside
// [0, E) are left out of the row, not of the sum.
constexpr int kRouteWaves = 4;
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_grad(const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ w,
                                                                 const float* __restrict__ dw, int64_t tokens, int E,
                                                                 int k, float* __restrict__ dlogits) {
  __shared__ float row[kRouteWaves][kMaxExperts];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  float* r = row[wv];
  // the wave's LDS accesses before it are complete for its other lanes after it
  auto wave_sync = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  for (int64_t t0 = (int64_t)blockIdx.x * kRouteWaves; t0 < tokens; t0 += (int64_t)gridDim.x * kRouteWaves) {
    const int64_t t = t0 + wv;
    if (t < tokens) {
      float s = 0.f;
      for (int j = lane; j < k; j += 64) s = fmaf(w[t * k + j], dw[t * k + j], s);
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
      for (int e = lane; e < E; e += 64) r[e] = 0.f;
      wave_sync();
      for (int j = lane; j < k; j += 64) {
        const int32_t e = ids[t * k + j];
        if (e >= 0 && e < E) atomicAdd(&r[e], w[t * k + j] * (dw[t * k + j] - s));
      }
      wave_sync();
      for (int e = lane; e < E; e += 64) dlogits[t * E + e] = r[e];
      wave_sync();
    }
  }
}

// ------------------------------------------------------------ host side ---

bool src_ok(moe_src_t d) { return d == MOE_SRC_BF16 || d == MOE_SRC_FP32; }
int64_t elem_size(moe_src_t d) { return d == MOE_SRC_BF16 ? 2 : 4; }
bool aligned(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }
// a row matrix that 16-byte pieces can walk
bool pieces16(const void* p, int64_t ld, int64_t es) { return aligned(p, 16) && ld * es % 16 == 0; }

// Sizes every dispatch operator shares.
moe_status_t check_sizes(moe_src_t dtype, int32_t T, int32_t H, int32_t k) {
  if (!src_ok(dtype) || T < 0 || H < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * k > (int64_t)1 << 30 || H > 1 << 24) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// a row matrix argument: present, element-aligned, rows at least H apart
bool matrix_ok(const void* p, int64_t ld, int32_t H, moe_src_t dtype) {
  return p && ld >= H && aligned(p, elem_size(dtype));
}

moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

template <typename T, int V>
void launch_gather_sum(const void* rows, int64_t rows_ld, int32_t num_rows, const int32_t* row_of, const float* w,
                       int32_t T_, int32_t H, int32_t k, const void* residual, int64_t res_ld, void* y, int64_t y_ld,
                       hipStream_t st) {
  RowMap m = row_map(T_, H / V);
  const bool stream = (int64_t)T_ * H * (int64_t)sizeof(T) >= kStreamBytes;
  // several pieces per thread: 16-byte ones in large calls, elements where that
  // leaves enough workgroups
  constexpr int U = V == 1 ? 4 : 2;
  const bool more = m.cblocks >= U && (V == 1 ? m.nblocks >= kElementBlocks : stream);
  if (more) m = with_pieces(m, U);
  const unsigned g = grid_blocks(m.nblocks);
#define MOE_GATHER_SUM(W, S, U)                                                                               \
  k_gather_sum<T, V, W, S, U><<<g, kThreadsD, 0, st>>>(m, (const T*)rows, rows_ld, num_rows, row_of, w, k,    \
                                                       (const T*)residual, res_ld, (T*)y, y_ld)
  constexpr bool S = V > 1;  // (elements are not stored past the caches)
  if (w && more) MOE_GATHER_SUM(true, S, U);
  else if (w && stream && S) MOE_GATHER_SUM(true, S, 1);
  else if (w) MOE_GATHER_SUM(true, false, 1);
  else if (more) MOE_GATHER_SUM(false, S, U);
  else if (stream && S) MOE_GATHER_SUM(false, S, 1);
  else MOE_GATHER_SUM(false, false, 1);
#undef MOE_GATHER_SUM
}

// moe_unpermute, and with w and residual null the gradient of moe_permute
moe_status_t gather_sum(const void* rows, moe_src_t dtype, int64_t rows_ld, int32_t num_rows, const int32_t* row_of,
                        const float* w, int32_t T, int32_t H, int32_t k, const void* residual, int64_t res_ld,
                        void* y, int64_t y_ld, hipStream_t stream) {
  moe_status_t a = check_arch();
  if (a != MOE_OK) return a;
  const int64_t es = elem_size(dtype);
  const bool vec = (int64_t)H * es % 16 == 0 && pieces16(y, y_ld, es) && (num_rows == 0 || pieces16(rows, rows_ld, es)) &&
                   (!residual || pieces16(residual, res_ld, es));
  if (dtype == MOE_SRC_BF16) {
    if (vec) launch_gather_sum<__bf16, 8>(rows, rows_ld, num_rows, row_of, w, T, H, k, residual, res_ld, y, y_ld, stream);
    else launch_gather_sum<__bf16, 1>(rows, rows_ld, num_rows, row_of, w, T, H, k, residual, res_ld, y, y_ld, stream);
  } else {
    if (vec) launch_gather_sum<float, 4>(rows, rows_ld, num_rows, row_of, w, T, H, k, residual, res_ld, y, y_ld, stream);
    else launch_gather_sum<float, 1>(rows, rows_ld, num_rows, row_of, w, T, H, k, residual, res_ld, y, y_ld, stream);
  }
  return launched();
}

}  // namespace

}  // namespace moe_mx

using namespace moe_mx;

// ------------------------------------------------------- public entry points

extern "C" moe_status_t moe_permute(const void* x, moe_src_t dtype, int64_t x_ld, int32_t T, int32_t H, int32_t E,
                                    int32_t k, const int32_t* expert_offsets, const int32_t* sorted_assign,
                                    int32_t local_expert_offset, int32_t local_num_experts, void* rows,
                                    int64_t rows_ld, int32_t num_rows, int32_t* row_of, hipStream_t stream) {
  moe_status_t v = check_sizes(dtype, T, H, k);
  if (v != MOE_OK) return v;
  if (E < 1 || E > kMaxExperts || k > E || num_rows < 0) return MOE_ERR_INVALID_ARG;
  const int32_t n = local_num_experts == 0 ? E : local_num_experts;
  if (local_expert_offset < 0 || n < 0 || (int64_t)local_expert_offset + n > E) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!expert_offsets || !sorted_assign || !row_of || !matrix_ok(x, x_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && !matrix_ok(rows, rows_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  moe_status_t a = check_arch();
  if (a != MOE_OK) return a;
  const int64_t es = elem_size(dtype), A = (int64_t)T * k;
  const bool vec = (int64_t)H * es % 16 == 0 && pieces16(x, x_ld, es) && (num_rows == 0 || pieces16(rows, rows_ld, es));
  const int V = vec ? (int)(16 / es) : 1;
  if (A * H * es >= kTokenBytes) {
    // row_of first, then each token's row read once and written to its rows
    const RowMap mt = row_map(T, H / V);
    const unsigned gi = grid_blocks((A + kThreadsD - 1) / kThreadsD), gt = grid_blocks(mt.nblocks);
    k_invert<<<gi, kThreadsD, 0, stream>>>(A, expert_offsets, sorted_assign, local_expert_offset, n, num_rows, row_of);
#define MOE_PERMUTE_TOKENS(P)                                                                                       \
  k_permute_tokens<P><<<gt, kThreadsD, 0, stream>>>(mt, (const P*)x, x_ld / V, k, row_of, (P*)rows, rows_ld / V,    \
                                                    num_rows)
    if (vec) MOE_PERMUTE_TOKENS(uint4);
    else if (dtype == MOE_SRC_BF16) MOE_PERMUTE_TOKENS(uint16_t);
    else MOE_PERMUTE_TOKENS(uint32_t);
#undef MOE_PERMUTE_TOKENS
    return launched();
  }
  RowMap m = row_map(A, H / V);
  // four elements per thread where that leaves enough workgroups (1024 x 4095 bf16,
  // k = 4: 20 us against 46)
  const bool more = !vec && m.cblocks >= 4 && m.nblocks >= kElementBlocks;
  if (more) m = with_pieces(m, 4);
  const unsigned g = grid_blocks(m.nblocks);
#define MOE_PERMUTE_ROWS(P, U)                                                                                      \
  k_permute_rows<P, U><<<g, kThreadsD, 0, stream>>>(m, (const P*)x, x_ld / V, k, expert_offsets, sorted_assign,     \
                                                    local_expert_offset, n, (P*)rows, rows_ld / V, num_rows, row_of)
  if (vec) MOE_PERMUTE_ROWS(uint4, 1);
  else if (dtype == MOE_SRC_BF16 && more) MOE_PERMUTE_ROWS(uint16_t, 4);
  else if (dtype == MOE_SRC_BF16) MOE_PERMUTE_ROWS(uint16_t, 1);
  else if (more) MOE_PERMUTE_ROWS(uint32_t, 4);
  else MOE_PERMUTE_ROWS(uint32_t, 1);
#undef MOE_PERMUTE_ROWS
  return launched();
}

extern "C" moe_status_t moe_permute_backward(const void* drows, moe_src_t dtype, int64_t drows_ld, int32_t num_rows,
                                             const int32_t* row_of, int32_t T, int32_t H, int32_t k, void* dx,
                                             int64_t dx_ld, hipStream_t stream) {
  moe_status_t v = check_sizes(dtype, T, H, k);
  if (v != MOE_OK) return v;
  if (num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!row_of || !matrix_ok(dx, dx_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && !matrix_ok(drows, drows_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  return gather_sum(drows, dtype, drows_ld, num_rows, row_of, nullptr, T, H, k, nullptr, 0, dx, dx_ld, stream);
}

extern "C" moe_status_t moe_unpermute(const void* rows, moe_src_t dtype, int64_t rows_ld, int32_t num_rows,
                                      const int32_t* row_of, const float* topk_w, int32_t T, int32_t H, int32_t k,
                                      const void* residual, int64_t residual_ld, void* y, int64_t y_ld,
                                      hipStream_t stream) {
  moe_status_t v = check_sizes(dtype, T, H, k);
  if (v != MOE_OK) return v;
  if (num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!row_of || !topk_w || !matrix_ok(y, y_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && !matrix_ok(rows, rows_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (residual && !matrix_ok(residual, residual_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  return gather_sum(rows, dtype, rows_ld, num_rows, row_of, topk_w, T, H, k, residual, residual_ld, y, y_ld, stream);
}

// A workgroup takes a token with all of its slots, so that dy is read once (4096 x
// 2048 bf16, k = 6: 43 us, 50 with a workgroup per slot).  Otherwise one per slot:
// a wave where rows are narrow and four would mostly wait for their sums (4096 x 864
// bf16, k = 8: 31 us against 45; 4096 x 267, k = 4: 10 against 18), and where there are
// few tokens 256 threads (64 x 2048, k = 6: 4.8 against 6.0) or, for rows of two pieces
// per thread and more, 1024 (64 x 27392, k = 3: 7 against 24; 11 x 7168, k = 8: 4.9
// against 10.6).  From 1024 tokens of 2048 or more values on the first is as fast.
constexpr int kNarrowRow = 1024;  // values
constexpr int kFewTokens = 256;
template <typename T, int V>
static void launch_unpermute_grad(const void* dy, int64_t dy_ld, const void* rows, int64_t rows_ld, int32_t num_rows,
                                  const int32_t* row_of, const float* w, int32_t tokens, int32_t H, int32_t k,
                                  void* drows, int64_t drows_ld, float* dw, hipStream_t st) {
#define MOE_UNPERMUTE_GRAD(S, TH, Q)                                                                               \
  k_unpermute_grad<T, V, S, TH, Q><<<grid_blocks((int64_t)tokens * ((k + Q - 1) / Q)), TH, 0, st>>>(               \
      tokens, H / V, (const T*)dy, dy_ld, (const T*)rows, rows_ld, num_rows, row_of, w, k, (T*)drows, drows_ld, dw)
  const bool stream = (int64_t)tokens * H * (int64_t)sizeof(T) >= kStreamBytes;
  if (H <= kNarrowRow) {
    if (stream) MOE_UNPERMUTE_GRAD(true, 64, 1);
    else MOE_UNPERMUTE_GRAD(false, 64, 1);
  } else if (tokens <= kFewTokens) {
    if (H / V >= 2 * 1024) MOE_UNPERMUTE_GRAD(false, 1024, 1);
    else MOE_UNPERMUTE_GRAD(false, kThreadsD, 1);
  } else {
    if (stream) MOE_UNPERMUTE_GRAD(true, kThreadsD, kSlots);
    else MOE_UNPERMUTE_GRAD(false, kThreadsD, kSlots);
  }
#undef MOE_UNPERMUTE_GRAD
}

extern "C" moe_status_t moe_unpermute_backward(const void* dy, moe_src_t dtype, int64_t dy_ld, const void* rows,
                                               int64_t rows_ld, int32_t num_rows, const int32_t* row_of,
                                               const float* topk_w, int32_t T, int32_t H, int32_t k, void* drows,
                                               int64_t drows_ld, float* dw, hipStream_t stream) {
  moe_status_t v = check_sizes(dtype, T, H, k);
  if (v != MOE_OK) return v;
  if (num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!row_of || !topk_w || !dw || !matrix_ok(dy, dy_ld, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && (!matrix_ok(rows, rows_ld, H, dtype) || !matrix_ok(drows, drows_ld, H, dtype)))
    return MOE_ERR_INVALID_ARG;
  moe_status_t a = check_arch();
  if (a != MOE_OK) return a;
  const int64_t es = elem_size(dtype);
  const bool vec = (int64_t)H * es % 16 == 0 && pieces16(dy, dy_ld, es) &&
                   (num_rows == 0 || (pieces16(rows, rows_ld, es) && pieces16(drows, drows_ld, es)));
  if (dtype == MOE_SRC_BF16) {
    if (vec) launch_unpermute_grad<__bf16, 8>(dy, dy_ld, rows, rows_ld, num_rows, row_of, topk_w, T, H, k, drows, drows_ld, dw, stream);
    else launch_unpermute_grad<__bf16, 1>(dy, dy_ld, rows, rows_ld, num_rows, row_of, topk_w, T, H, k, drows, drows_ld, dw, stream);
  } else {
    if (vec) launch_unpermute_grad<float, 4>(dy, dy_ld, rows, rows_ld, num_rows, row_of, topk_w, T, H, k, drows, drows_ld, dw, stream);
    else launch_unpermute_grad<float, 1>(dy, dy_ld, rows, rows_ld, num_rows, row_of, topk_w, T, H, k, drows, drows_ld, dw, stream);
  }
  return launched();
}

extern "C" moe_status_t moe_route_backward(const int32_t* topk_ids, const float* topk_w, const float* dw, int32_t T,
                                           int32_t E, int32_t k, float* dlogits, hipStream_t stream) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * k > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!topk_ids || !topk_w || !dw || !dlogits) return MOE_ERR_INVALID_ARG;
  moe_status_t a = check_arch();
  if (a != MOE_OK) return a;
  k_route_grad<<<grid_blocks(((int64_t)T + kRouteWaves - 1) / kRouteWaves), 64 * kRouteWaves, 0, stream>>>(
      topk_ids, topk_w, dw, T, E, k, dlogits);
  return launched();
}
