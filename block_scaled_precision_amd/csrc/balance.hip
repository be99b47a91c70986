// Balance of the router: moe_balance (load-balance loss, z-loss and tokens per
// expert of every sequence of a packed batch) and its gradient, next to moe_route
// and moe_route_backward (TokenSpeed SiTU page, "Supported contract": global top-k
// ids over a routed batch).
//
// With p[t] the softmax of a counted token's logits and lse[t] their log-sum-exp,
// n_s the counted tokens of sequence s, S' the sequences that have one, n their sum:
//   balance = E / S' sum_s sum_e (counts[s, e] / (k n_s)) (sum_{t in s} p[t, e] / n_s)
//   z       = 1 / n sum_t lse[t]^2
//   dlogits[t, e] = d_balance E / (S' n_s) p_e (f_e - sum_j f_j p_j)
//                   + d_z 2 / n lse[t] p_e,     f_e = counts[s, e] / (k n_s)
// counts take no gradient (the choice of experts is piecewise constant), and since p =
// exp(logit - lse), the gradient needs one pass over the logits and no second pass
// over what the loss computed.
//
// Both directions are bound by reading the logits once (and writing their gradient
// once).  A row is held in registers by a group of 16, 32 or 64 neighbouring lanes,
// pieces of 16 bytes each where lengths, strides and addresses allow, single values
// elsewhere, so that a maximum and two sums over the group are all that a row costs.
// A loss over few tokens takes one launch of one workgroup.  Otherwise workgroups
// take chunks of consecutive rows and leave, for each sequence that a chunk meets,
// its sums in a slot; a second launch adds the slots in order, and the workgroup of it
// that is last to arrive adds up what the others left, in order again: no result
// depends on scheduling, and results repeat bit for bit.  Sums over the rows of a
// chunk are held in fp32, sums over chunks and sequences in fp64.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"

namespace moe_mx {

namespace {

constexpr int kThreadsB = 256;
constexpr int kOneThreads = 1024;
constexpr float kNegInf = -__builtin_inff();

typedef float v4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------- rows in registers --

template <int CTRL> __device__ __forceinline__ float dpp_mov(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Reduction over a group of L neighbouring lanes; every lane gets the same bits.
template <int L, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  v = op(v, dpp_mov<0xb1>(v));   // quad_perm 1,0,3,2
  v = op(v, dpp_mov<0x4e>(v));   // quad_perm 2,3,0,1
  v = op(v, dpp_mov<0x141>(v));  // row_half_mirror
  v = op(v, dpp_mov<0x140>(v));  // row_mirror
  if (L >= 32) v = op(v, __shfl_xor(v, 16));
  if (L >= 64) v = op(v, __shfl_xor(v, 32));
  return v;
}
struct Sum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
// (NaN counts as +inf: a row with one is not empty, and its sums are NaN)
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// P pieces of V values of a row, piece q of lane c at value (q L + c) V.
template <int V, int P> struct RowRegs {
  float v[P * V];
};
template <int V, int L, int P>
__device__ __forceinline__ void load_row(RowRegs<V, P>& r, const float* row, int E, int c, float fill) {
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const int e = (q * L + c) * V;
    if constexpr (V == 4) {
      v4 x = {fill, fill, fill, fill};
      if (e < E) x = *(const v4*)(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[4 * q + i] = x[i];
    } else {
      r.v[q] = e < E ? row[e] : fill;
    }
  }
}

// Largest value, NaN taken as +inf (v == v fails for it)
template <int L, int N>
__device__ __forceinline__ float row_max(const float (&v)[N]) {
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, v[i] == v[i] ? v[i] : -kNegInf);
  return group_reduce<L>(m, Max());
}

// -------------------------------------------------------------- sequences --

// Rows [lo, hi) of sequence s, within [0, T)
__device__ __forceinline__ void seq_rows(const int32_t* off, int s, int T, int& lo, int& hi) {
  if (!off) {
    lo = 0;
    hi = T;
    return;
  }
  lo = min(max(off[s], 0), T);
  hi = min(max(off[s + 1], lo), T);
}
// The last sequence that begins at or before row t, 0 if none does
template <class Off>
__device__ __forceinline__ int seq_search(Off off, int S, int t) {
  int lo = 0, hi = S;  // begins[lo] <= t < begins[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off(mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- forward --

struct BalanceArgs {
  const float* logits;
  int64_t ld;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* off;
  int T, E, k, S;
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  float* lse;
  // slots chunk + sequence of the chunks' sums (a chunk and a sequence that meet
  // never share one with another pair, as both only go up), and what the
  // second launch leaves
  int rows, chunks;       // rows per chunk, chunks
  float* sum_p;           // [chunks + S, E]
  int32_t* sum_c;         // [chunks + S, E]
  float* sum_z;           // [chunks + S]
  int32_t* sum_n;         // [chunks + S]
  double* part;           // [S, blocks]
  double* part_z;         // [S]
  uint32_t* arrived;
};

// What a workgroup of TH threads gathers of the rows [lo, hi) of one sequence
template <int V, int L, int P, int TH> struct Gathered {
  static constexpr int GROUPS = TH / L;
  float p[GROUPS][V * L * P];  // one row of sums per group (GROUPS V L P <= 16 KiB of them)
  int32_t c[kMaxExperts];
  float z[GROUPS];
  int32_t n[GROUPS];
};

// Rows [lo, hi): their lse, and into g each group's sums of p, lse^2 and tokens
// and all groups' counts.  g.c is zero at the start.
template <int V, int L, int P, int TH>
__device__ __forceinline__ void gather_rows(const BalanceArgs& a, int lo, int hi, Gathered<V, L, P, TH>& g) {
  constexpr int G = TH / L;
  const int c = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  float acc[P * V];
#pragma unroll
  for (int i = 0; i < P * V; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  for (int t = lo + grp; t < hi; t += G) {
    RowRegs<V, P> r;
    load_row<V, L, P>(r, a.logits + (int64_t)t * a.ld, a.E, c, kNegInf);
    const int32_t id0 = c < a.k ? a.ids[(int64_t)t * a.k + c] : -1;
    const bool live = !a.mask || a.mask[t] != 0;
    const float m = row_max<L>(r.v);
    const bool counted = live && m != kNegInf;
    if (!counted) {
      if (c == 0) a.lse[t] = kNegInf;
      continue;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < P * V; ++i) {
      r.v[i] = expf(r.v[i] - m);
      s += r.v[i];
    }
    s = group_reduce<L>(s, Sum());
    const float inv = 1.0f / s, l = m + logf(s);
#pragma unroll
    for (int i = 0; i < P * V; ++i) acc[i] = fmaf(r.v[i], inv, acc[i]);
    if (id0 >= 0 && id0 < a.E) atomicAdd(&g.c[id0], 1);
    for (int j = c + L; j < a.k; j += L) {
      const int32_t id = a.ids[(int64_t)t * a.k + j];
      if (id >= 0 && id < a.E) atomicAdd(&g.c[id], 1);
    }
    z = fmaf(l, l, z);
    ++n;
    if (c == 0) a.lse[t] = l;
  }
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) g.p[grp][(q * L + c) * V + i] = acc[q * V + i];
  if (c == 0) {
    g.z[grp] = z;
    g.n[grp] = n;
  }
}

template <int V, int L, int P>
__global__ __launch_bounds__(kThreadsB) void k_balance_rows(BalanceArgs a) {
  using Gt = Gathered<V, L, P, kThreadsB>;
  __shared__ Gt g;
  const int t0 = blockIdx.x * a.rows, t1 = min(a.T, t0 + a.rows);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.arrived = 0;
  auto begins = [&](int i) { return a.off[i]; };
  int lo0 = 0, hi0 = a.T;
  if (a.off) {
    lo0 = min(max(a.off[0], 0), a.T);
    hi0 = min(max(a.off[a.S], 0), a.T);
    // rows of no sequence
    for (int t = t0 + threadIdx.x; t < t1; t += kThreadsB)
      if (t < lo0 || t >= hi0) a.lse[t] = kNegInf;
  }
  int t = max(t0, lo0);
  int s = a.off && t < t1 ? seq_search(begins, a.S, t) : 0;
  while (t < min(t1, hi0)) {
    int lo, hi;
    seq_rows(a.off, s, a.T, lo, hi);
    const int end = min(t1, hi);
    if (end <= t) break;  // offsets that do not ascend
    for (int e = threadIdx.x; e < a.E; e += kThreadsB) g.c[e] = 0;
    __syncthreads();
    gather_rows<V, L, P, kThreadsB>(a, t, end, g);
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < a.E; e += kThreadsB) {
      float p = 0.f;
#pragma unroll
      for (int q = 0; q < Gt::GROUPS; ++q) p += g.p[q][e];
      a.sum_p[slot * a.E + e] = p;
      a.sum_c[slot * a.E + e] = g.c[e];
    }
    if (threadIdx.x == 0) {
      float z = 0.f;
      int n = 0;
      for (int q = 0; q < Gt::GROUPS; ++q) {
        z += g.z[q];
        n += g.n[q];
      }
      a.sum_z[slot] = z;
      a.sum_n[slot] = n;
    }
    __syncthreads();
    t = end;
    if (t < min(t1, hi0)) s = seq_search(begins, a.S, t);
  }
}

// Sum over a workgroup's threads, in every thread; the order is fixed.  sh: a value
// per wave.
template <int TH, class T>
__device__ __forceinline__ T block_sum(T v, T* sh) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = sh[0];
#pragma unroll
  for (int w = 1; w < TH / 64; ++w) s += sh[w];
  return s;
}

// One workgroup per kFinishCols experts and sequence: 16 lanes along the
// experts, 16 along the sequence's chunks.
constexpr int kFinishCols = 16, kFinishChunks = kThreadsB / kFinishCols;
__global__ __launch_bounds__(kThreadsB) void k_balance_finish(BalanceArgs a) {
  __shared__ double sp[kFinishChunks][kFinishCols];
  __shared__ int32_t scn[kFinishChunks][kFinishCols];
  __shared__ double sh[kThreadsB / 64];
  __shared__ int32_t shi[kThreadsB / 64];
  __shared__ int32_t last;
  const int nb = (a.E + kFinishCols - 1) / kFinishCols;
  const int s = blockIdx.x / nb, b = blockIdx.x % nb;
  const int col = threadIdx.x % kFinishCols, ch = threadIdx.x / kFinishCols, e = b * kFinishCols + col;
  int lo, hi;
  seq_rows(a.off, s, a.T, lo, hi);
  const int c0 = lo / a.rows, c1 = hi > lo ? (hi - 1) / a.rows + 1 : c0;
  double p = 0.0;
  int32_t cnt = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int c = c0 + ch; c < c1; c += kFinishChunks) {
      const int64_t i = ((int64_t)c + s) * a.E + e;
      p += (double)a.sum_p[i];
      cnt += a.sum_c[i];
    }
  }
  int32_t n = 0;
  double z = 0.0;
  for (int c = c0 + threadIdx.x; c < c1; c += kThreadsB) {
    n += a.sum_n[c + s];
    z += (double)a.sum_z[c + s];
  }
  sp[ch][col] = p;
  scn[ch][col] = cnt;
  n = block_sum<kThreadsB>(n, shi);
  double term = 0.0;
  if (threadIdx.x < kFinishCols && e < a.E) {
    p = 0.0;
    cnt = 0;
#pragma unroll
    for (int q = 0; q < kFinishChunks; ++q) {
      p += sp[q][col];
      cnt += scn[q][col];
    }
    a.counts[(int64_t)s * a.E + e] = cnt;
    if (n > 0) term = (double)cnt * p / ((double)a.k * n * n);
  }
  term = block_sum<kThreadsB>(term, sh);
  if (b == 0) {
    z = block_sum<kThreadsB>(z, sh);
    if (threadIdx.x == 0) {
      a.tokens[s] = n;
      a.part_z[s] = z;
    }
  }
  if (threadIdx.x == 0) {
    a.part[blockIdx.x] = term;
    __threadfence();
    last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();  // the other workgroups' sums, across the dies' caches
  double balance = 0.0, zs = 0.0;
  int32_t total = 0, used = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x; i += kThreadsB) balance += a.part[i];
  for (int i = threadIdx.x; i < a.S; i += kThreadsB) {
    const int32_t m = a.tokens[i];
    zs += a.part_z[i];
    total += m;
    used += m > 0;
  }
  balance = block_sum<kThreadsB>(balance, sh);
  zs = block_sum<kThreadsB>(zs, sh);
  total = block_sum<kThreadsB>(total, shi);
  used = block_sum<kThreadsB>(used, shi);
  if (threadIdx.x == 0) {
    a.tokens[a.S] = total;
    a.tokens[a.S + 1] = used;
    a.loss[0] = (float)(used > 0 ? balance * a.E / used : 0.0);
    a.loss[1] = (float)(total > 0 ? zs / total : 0.0);
  }
}

// All of it in one workgroup, one sequence after the other
template <int V, int L, int P>
__global__ __launch_bounds__(kOneThreads) void k_balance_one(BalanceArgs a) {
  using Gt = Gathered<V, L, P, kOneThreads>;
  __shared__ Gt g;
  __shared__ double sh[kOneThreads / 64];
  __shared__ int32_t shi[kOneThreads / 64];
  double balance = 0.0, zs = 0.0;
  int total = 0, used = 0;
  if (a.off) {
    const int lo0 = min(max(a.off[0], 0), a.T), hi0 = min(max(a.off[a.S], 0), a.T);
    for (int t = threadIdx.x; t < a.T; t += kOneThreads)
      if (t < lo0 || t >= hi0) a.lse[t] = kNegInf;
  }
  for (int s = 0; s < a.S; ++s) {
    int lo, hi;
    seq_rows(a.off, s, a.T, lo, hi);
    for (int e = threadIdx.x; e < a.E; e += kOneThreads) g.c[e] = 0;
    __syncthreads();
    gather_rows<V, L, P, kOneThreads>(a, lo, hi, g);
    __syncthreads();
    const int n = block_sum<kOneThreads>(threadIdx.x < Gt::GROUPS ? g.n[threadIdx.x] : 0, shi);
    const double z = block_sum<kOneThreads>(threadIdx.x < Gt::GROUPS ? (double)g.z[threadIdx.x] : 0.0, sh);
    double term = 0.0;
    for (int e = threadIdx.x; e < a.E; e += kOneThreads) {
      const int32_t cnt = g.c[e];
      a.counts[(int64_t)s * a.E + e] = cnt;
      double p = 0.0;
#pragma unroll 8
      for (int q = 0; q < Gt::GROUPS; ++q) p += (double)g.p[q][e];
      if (n > 0) term += (double)cnt * p / ((double)a.k * n * n);
    }
    term = block_sum<kOneThreads>(term, sh);
    balance += term;
    zs += z;
    total += n;
    used += n > 0;
    if (threadIdx.x == 0) a.tokens[s] = n;
  }
  if (threadIdx.x == 0) {
    a.tokens[a.S] = total;
    a.tokens[a.S + 1] = used;
    a.loss[0] = (float)(used > 0 ? balance * a.E / used : 0.0);
    a.loss[1] = (float)(total > 0 ? zs / total : 0.0);
  }
}

// --------------------------------------------------------------- backward --

struct BalanceGradArgs {
  const float* dloss;
  const float* logits;
  int64_t ld;
  const int32_t* counts;
  const int32_t* tokens;
  const float* lse;
  const int32_t* off;
  int T, E, k, S;
  int per;                // consecutive rows per group
  const float* add;
  int64_t add_ld;
  float* dlogits;
  int64_t dlogits_ld;
};

constexpr int kSeqLds = 1024;  // offsets that are searched in LDS

// A group of L lanes takes `per` consecutive rows, so that the f of their sequence
// stay in registers from row to row.  STREAM: the gradient and what is added to it
// bypass the caches' retention.
template <int V, int L, int P, bool STREAM>
__global__ __launch_bounds__(kThreadsB) void k_balance_grad(BalanceGradArgs a) {
  __shared__ int32_t soff[kSeqLds + 1];
  const int c = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const bool in_lds = a.off && a.S <= kSeqLds;
  if (in_lds) {
    for (int i = threadIdx.x; i <= a.S; i += kThreadsB) soff[i] = a.off[i];
    __syncthreads();
  }
  auto begins = [&](int i) { return in_lds ? soff[i] : a.off[i]; };
  const float d0 = a.dloss[0], d1 = a.dloss[1];
  const int total = a.tokens[a.S], used = a.tokens[a.S + 1];
  const float kz = total > 0 ? d1 * (2.0f / (float)total) : 0.f;
  const float kb = used > 0 ? d0 * ((float)a.E / (float)used) : 0.f;
  int seq = -1;
  float f[P * V], ks = 0.f;
  const int64_t r0 = ((int64_t)blockIdx.x * (kThreadsB / L) + grp) * a.per;
  const int r1 = (int)min((int64_t)a.T, r0 + a.per);
  for (int t = (int)min(r0, (int64_t)a.T); t < r1; ++t) {
    RowRegs<V, P> r, ad;
    load_row<V, L, P>(r, a.logits + (int64_t)t * a.ld, a.E, c, kNegInf);
    const float l = a.lse[t];
    if (a.add) {
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int e = (q * L + c) * V;
        const float* src = a.add + (int64_t)t * a.add_ld + e;
        if constexpr (V == 4) {
          v4 x = {0.f, 0.f, 0.f, 0.f};
          if (e < a.E) x = STREAM ? __builtin_nontemporal_load((const v4*)src) : *(const v4*)src;
#pragma unroll
          for (int i = 0; i < 4; ++i) ad.v[4 * q + i] = x[i];
        } else {
          ad.v[q] = e < a.E ? *src : 0.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < P * V; ++i) ad.v[i] = 0.f;
    }
    if (l != kNegInf) {
      const int s = !a.off ? 0 : seq >= 0 && t < begins(seq + 1) ? seq : seq_search(begins, a.S, t);
      if (s != seq) {
        seq = s;
        const int n = a.tokens[s];
        const float per = 1.0f / (float)max(n, 1), per_k = per / (float)a.k;
        ks = kb * per;
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int e = (q * L + c) * V + i;
            f[q * V + i] = e < a.E ? (float)a.counts[(int64_t)s * a.E + e] * per_k : 0.f;
          }
      }
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < P * V; ++i) {
        r.v[i] = expf(r.v[i] - l);
        dot = fmaf(f[i], r.v[i], dot);
      }
      dot = group_reduce<L>(dot, Sum());
      const float zl = kz * l;
#pragma unroll
      for (int i = 0; i < P * V; ++i) ad.v[i] = fmaf(r.v[i], fmaf(ks, f[i] - dot, zl), ad.v[i]);
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int e = (q * L + c) * V;
      if (e >= a.E) continue;
      float* dst = a.dlogits + (int64_t)t * a.dlogits_ld + e;
      if constexpr (V == 4) {
        const v4 x = {ad.v[4 * q], ad.v[4 * q + 1], ad.v[4 * q + 2], ad.v[4 * q + 3]};
        if constexpr (STREAM) __builtin_nontemporal_store(x, (v4*)dst);
        else *(v4*)dst = x;
      } else {
        *dst = ad.v[q];
      }
    }
  }
}

// ------------------------------------------------------------------- host --

constexpr int kMaxChunks = 512;
// Tokens up to which the loss takes one launch of one workgroup, for up to
// kOneSeqs sequences
constexpr int kOneTokens = 128, kOneSeqs = 4;

// Lanes per row and pieces per lane: calls F with them as compile-time constants.
template <class F>
void for_row_shape(bool vec, int E, F f) {
#define MOE_ROW_SHAPE(V, L, P) \
  if (E <= V * L * P) return f(std::integral_constant<int, V>(), std::integral_constant<int, L>(), \
                               std::integral_constant<int, P>())
  if (vec) {
    MOE_ROW_SHAPE(4, 16, 1);
    MOE_ROW_SHAPE(4, 32, 1);
    MOE_ROW_SHAPE(4, 16, 3);
    MOE_ROW_SHAPE(4, 32, 2);
    MOE_ROW_SHAPE(4, 32, 3);
    MOE_ROW_SHAPE(4, 64, 2);
    MOE_ROW_SHAPE(4, 64, 3);
    MOE_ROW_SHAPE(4, 64, 4);
  } else {
    MOE_ROW_SHAPE(1, 16, 1);
    MOE_ROW_SHAPE(1, 32, 1);
    MOE_ROW_SHAPE(1, 64, 1);
    MOE_ROW_SHAPE(1, 64, 2);
    MOE_ROW_SHAPE(1, 64, 4);
    MOE_ROW_SHAPE(1, 64, 8);
    MOE_ROW_SHAPE(1, 64, 16);
  }
#undef MOE_ROW_SHAPE
}

struct BalancePlan {
  bool one;
  int rows, chunks;
  size_t sum_p, sum_c, sum_z, sum_n, part, part_z, arrived, total;
};

BalancePlan balance_plan(int32_t T, int32_t E, int32_t S) {
  BalancePlan f = {};
  f.one = T <= kOneTokens && S <= kOneSeqs;
  if (f.one) return f;
  // chunks of whole rounds of a workgroup's groups (16 of them at most)
  f.rows = (int)align_up(std::max<size_t>(((size_t)T + kMaxChunks - 1) / kMaxChunks, 1), 16);
  f.chunks = (T + f.rows - 1) / f.rows;
  const size_t slots = (size_t)f.chunks + S;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = align_up(o + bytes, 256);
    return r;
  };
  f.sum_p = take(slots * E * 4);
  f.sum_c = take(slots * E * 4);
  f.sum_z = take(slots * 4);
  f.sum_n = take(slots * 4);
  f.part = take((size_t)S * ((E + kFinishCols - 1) / kFinishCols) * 8);
  f.part_z = take((size_t)S * 8);
  f.arrived = take(4);
  f.total = o;
  return f;
}

bool sizes_valid(int32_t T, int32_t E, int32_t k, int32_t S) {
  return T >= 0 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= E && S >= 1;
}
bool sizes_supported(int32_t T, int32_t E, int32_t k, int32_t S) {
  return (int64_t)T * k <= (int64_t)1 << 30 && (int64_t)S * E <= (int64_t)1 << 30 && T <= 1 << 30;
}
bool aligned_b(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }
bool matrix16(const float* p, int64_t ld, int32_t E) { return aligned_b(p, 16) && ld % 4 == 0 && E % 4 == 0; }
moe_status_t launched_b() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Gradients from this size on are stored past the caches.
constexpr int64_t kStreamGrad = 16 << 20;

}  // namespace

}  // namespace moe_mx

using namespace moe_mx;

extern "C" size_t moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t S) {
  if (!sizes_valid(T, E, 1, S) || !sizes_supported(T, E, 1, S)) return 0;
  return balance_plan(T, E, S).total;
}

extern "C" moe_status_t moe_balance(const float* logits, int64_t logits_ld, const int32_t* topk_ids,
                                    const uint8_t* mask, const int32_t* seq_offsets, int32_t T, int32_t E, int32_t k,
                                    int32_t S, float* loss, int32_t* counts, int32_t* tokens, float* lse,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!sizes_valid(T, E, k, S) || (!seq_offsets && S != 1)) return MOE_ERR_INVALID_ARG;
  if (!sizes_supported(T, E, k, S)) return MOE_ERR_UNSUPPORTED;
  if (!loss || !counts || !tokens || !aligned_b(loss, 4) || !aligned_b(counts, 4) || !aligned_b(tokens, 4) ||
      !aligned_b(seq_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !lse || logits_ld < E || !aligned_b(logits, 4) || !aligned_b(topk_ids, 4) ||
                !aligned_b(lse, 4)))
    return MOE_ERR_INVALID_ARG;
  const BalancePlan f = balance_plan(T, E, S);
  if (f.total > 0 && (!workspace || workspace_bytes < f.total)) return MOE_ERR_WORKSPACE;
  if (f.total > 0 && !aligned_b(workspace, 256)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  BalanceArgs a = {};
  a.logits = logits;
  a.ld = logits_ld;
  a.ids = topk_ids;
  a.mask = mask;
  a.off = seq_offsets;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.lse = lse;
  const bool vec = T > 0 && matrix16(logits, logits_ld, E);
  if (f.one) {
    for_row_shape(vec, E, [&](auto V, auto L, auto P) {
      k_balance_one<V.value, L.value, P.value><<<1, kOneThreads, 0, stream>>>(a);
    });
    return launched_b();
  }
  char* ws = (char*)workspace;
  a.rows = f.rows;
  a.chunks = f.chunks;
  a.sum_p = (float*)(ws + f.sum_p);
  a.sum_c = (int32_t*)(ws + f.sum_c);
  a.sum_z = (float*)(ws + f.sum_z);
  a.sum_n = (int32_t*)(ws + f.sum_n);
  a.part = (double*)(ws + f.part);
  a.part_z = (double*)(ws + f.part_z);
  a.arrived = (uint32_t*)(ws + f.arrived);
  for_row_shape(vec, E, [&](auto V, auto L, auto P) {
    k_balance_rows<V.value, L.value, P.value><<<(unsigned)std::max(f.chunks, 1), kThreadsB, 0, stream>>>(a);
  });
  const moe_status_t r = launched_b();
  if (r != MOE_OK) return r;
  k_balance_finish<<<(unsigned)((int64_t)S * ((E + kFinishCols - 1) / kFinishCols)), kThreadsB, 0, stream>>>(a);
  return launched_b();
}

extern "C" moe_status_t moe_balance_backward(const float* dloss, const float* logits, int64_t logits_ld,
                                             const int32_t* counts, const int32_t* tokens, const float* lse,
                                             const int32_t* seq_offsets, int32_t T, int32_t E, int32_t k, int32_t S,
                                             const float* add, int64_t add_ld, float* dlogits, int64_t dlogits_ld,
                                             hipStream_t stream) {
  if (!sizes_valid(T, E, k, S) || (!seq_offsets && S != 1)) return MOE_ERR_INVALID_ARG;
  if (!sizes_supported(T, E, k, S)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dloss || !logits || !counts || !tokens || !lse || !dlogits || logits_ld < E || dlogits_ld < E ||
      (add && add_ld < E))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {(const void*)dloss, (const void*)logits, (const void*)counts, (const void*)tokens,
                        (const void*)lse, (const void*)seq_offsets, (const void*)add, (const void*)dlogits})
    if (!aligned_b(q, 4)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  BalanceGradArgs a = {dloss, logits, logits_ld, counts, tokens, lse, seq_offsets, T, E, k, S, 1,
                       add,   add_ld, dlogits,   dlogits_ld};
  const bool vec = matrix16(logits, logits_ld, E) && matrix16(dlogits, dlogits_ld, E) &&
                   (!add || matrix16(add, add_ld, E));
  const bool stream_out = (int64_t)T * E * 4 >= kStreamGrad;
  for_row_shape(vec, E, [&](auto V, auto L, auto P) {
    constexpr int G = kThreadsB / L.value;
    // rows per group: one where that leaves the chip room, more once there are
    // workgroups enough
    a.per = (int)std::min<int64_t>(16, std::max<int64_t>(1, (int64_t)T / (G * 2048)));
    const int64_t blocks = ((int64_t)T + (int64_t)G * a.per - 1) / ((int64_t)G * a.per);
    if (stream_out) k_balance_grad<V.value, L.value, P.value, true><<<(unsigned)blocks, kThreadsB, 0, stream>>>(a);
    else k_balance_grad<V.value, L.value, P.value, false><<<(unsigned)blocks, kThreadsB, 0, stream>>>(a);
  });
  return launched_b();
}
