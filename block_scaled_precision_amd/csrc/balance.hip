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
// counts take no gradient (the choice of experts is piecewise constant), and since p is
// exp(logit - lse) to within a factor of the row, the gradient needs one pass over the logits.
// The factor (lse's rounding, 2^-24 |lse| and more, and all of log E where |lse| is 2^26)
// goes with the sum of the row's exponentials, which is taken along with <f, p>.
//
// Both directions read the logits once (and write their gradient once).  A row is held in
// registers by a group of 16, 32 or 64 neighbouring lanes, pieces of 16 bytes each where
// lengths, strides and addresses allow, single values elsewhere, so that a maximum and a sum
// over the group are all that a row costs beside its values.
// A loss over few tokens takes one launch of one workgroup.  Otherwise workgroups
// take chunks of consecutive rows and leave, for each sequence that a chunk meets,
// its sums in a slot; a second launch adds the slots in order, and the workgroup of it
// that is last to arrive adds up what the others left, in order again: no result
// depends on scheduling, and results repeat bit for bit.  Sums over the rows of a
// chunk are held in fp32, sums over chunks and sequences in fp64.
//
// Measured (MI355X, warm; bytes at 5 TB/s in brackets): 65536 x 256 and what is added to its
// gradient 37 us [40]: bound by memory.  The loss is bound by what follows one after the
// other: 65536 x 128 13 + 6 us [7], 8192 x 384 in 13 sequences 7.5 + 7 [2.6], 64 x 384 7 in one
// launch, of which a launch that does nothing takes 2.  In the first launch of 65536 x 128 a wave
// waits for half of its 23700 cycles, as a chunk's rows come in two batches, load, compute, load,
// compute, and the 1625 vector instructions (25 a value) of the two waves of a SIMD take the
// other half; in the second and in small calls it is memory's latencies of about a microsecond.
// On the way there: the offsets through LDS and rows without regard to sequences 9.0 -> 7.5 us
// (8192 x 384), 16 lanes a row and a cheaper exponential 15.5 -> 12.5 (65536 x 128), no fences in
// the second launch 16.6 -> 11.3, fewer workgroups in it where there are many sequences -> 8.2,
// sums over lanes by register moves -> 7.
#include <hip/hip_runtime.h>

#include "balance_plan.h"
#include "copy_ring.h"
#include "internal.h"
#include "mx_device.h"

namespace moe_mx {

namespace {

constexpr int kOneThreads = 1024;
constexpr float kNegInf = -__builtin_inff();

typedef float v4 __attribute__((ext_vector_type(4)));

// A barrier for what lies in LDS: __syncthreads also waits for every store to memory, a
// microsecond each time.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  wait_lgkm0();
  barrier();
}

// ------------------------------------------------------- rows in registers --

// Reduction over a group of L neighbouring lanes; every lane gets the same bits.
template <int L, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  v = op(v, lane_move<0xb1>(v));   // quad_perm 1,0,3,2
  v = op(v, lane_move<0x4e>(v));   // quad_perm 2,3,0,1
  v = op(v, lane_move<0x141>(v));  // row_half_mirror
  v = op(v, lane_move<0x140>(v));  // row_mirror
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

// exp(d) for d <= 0, 0 for NaN: d log2(e) in two parts and the hardware's exp2, off by 1.3 |d| + 4
// half steps of fp32; a value below 2^-126 may become 0.  (7 instructions for expf's 12, of
// which the loss has little else.)
__device__ __forceinline__ float exp_below(float d) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
  d = fmaxf(d, -200.0f);
  const float t = d * kLog2e, rest = fmaf(d, kLog2e, -t);
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, rest * kLn2, e);
}

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

// Offsets of up to so many sequences are held in LDS: one load by all threads in place of a
// chain of them.
constexpr int kSeqLds = 1024;
struct Offsets {
  const int32_t* mem;
  const int32_t* lds;  // or nullptr
  __device__ __forceinline__ int operator()(int i) const { return lds ? lds[i] : mem[i]; }
};
template <int TH>
__device__ __forceinline__ Offsets load_offsets(const int32_t* off, int S, int32_t* lds) {
  if (!off || S > kSeqLds) return {off, nullptr};
  for (int i = threadIdx.x; i <= S; i += TH) lds[i] = off[i];
  lds_barrier();
  return {off, lds};
}
// Rows [lo, hi) of sequence s, within [0, T)
__device__ __forceinline__ void seq_rows(const Offsets& off, int s, int T, int& lo, int& hi) {
  if (!off.mem) {
    lo = 0;
    hi = T;
    return;
  }
  lo = min(max(off(s), 0), T);
  hi = min(max(off(s + 1), lo), T);
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
  int rows;               // per chunk
  float* sum_p;           // [chunks + S, E]
  int32_t* sum_c;         // [chunks + S, E]
  float* sum_z;           // [chunks + S]
  int32_t* sum_n;         // [chunks + S]
  double* part;           // [S, blocks]
  double* part_z;         // [S]
  uint32_t* arrived;
};

// What a workgroup of TH threads gathers of the rows of one sequence
template <int V, int L, int P, int TH> struct Gathered {
  static constexpr int GROUPS = TH / L;
  float p[GROUPS][V * L * P];  // one row of sums per group (4 TH V P bytes: 128 KiB at most)
  int32_t c[kMaxExperts];
  float z[GROUPS];
  int32_t n[GROUPS];
};

// Rows [t0, t1), which lie in sequences: their lse, and for each sequence s that they meet, in
// order, into g each group's sums of p, lse^2 and tokens and all groups' counts, and
// flush(s) between two barriers.  Rows are loaded and their softmax is taken without regard to
// the sequences, which a batch of rows may meet several of: a pass over the rows for each
// of them took 3 us more where one chunk met two.
template <int V, int L, int P, int TH, class Flush>
__device__ __forceinline__ void gather_rows(const BalanceArgs& a, const Offsets& off, int t0, int t1,
                                            Gathered<V, L, P, TH>& g, Flush flush) {
  if (t0 >= t1) return;
  constexpr int G = TH / L;
  // as many rows at once as 32 registers hold, up to 4: a load takes as long as all of them
  // (one where the whole loss has one workgroup, whose lanes cover most of its rows)
  constexpr int U = TH == kOneThreads ? 1 : P * V <= 8 ? 4 : P * V <= 16 ? 2 : 1;
  const int c = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  float acc[P * V], z = 0.f;
  int n = 0;
#pragma unroll
  for (int i = 0; i < P * V; ++i) acc[i] = 0.f;
  for (int e = threadIdx.x; e < a.E; e += TH) g.c[e] = 0;
  int t = t0, s = -1, end = t0;  // the first row that is not gathered, its sequence, where that ends
  for (int b = t0; b < t1; b += U * G) {
    RowRegs<V, P> rows[U];
    int32_t ids[U];
    float l[U], inv[U];
    bool counted[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = b + grp + u * G;
      const bool in = r < t1;
      load_row<V, L, P>(rows[u], a.logits + (int64_t)r * a.ld, in ? a.E : 0, c, kNegInf);
      ids[u] = in && c < a.k ? a.ids[(int64_t)r * a.k + c] : -1;
      counted[u] = in && (!a.mask || a.mask[r] != 0);
    }
    if (s < 0) {
      s = a.off ? seq_search(off, a.S, t) : 0;
      int lo;
      seq_rows(off, s, a.T, lo, end);
      lds_barrier();  // the counts are zero
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * G >= t1) break;
      const float m = row_max<L>(rows[u].v);
      counted[u] = counted[u] && m != kNegInf;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P * V; ++i) {
        rows[u].v[i] = exp_below(rows[u].v[i] - m);
        sum += rows[u].v[i];
      }
      sum = m < -kNegInf ? group_reduce<L>(sum, Sum()) : __builtin_nanf("");
      inv[u] = 1.0f / sum;
      l[u] = counted[u] ? m + logf(sum) : kNegInf;
      const int r = b + grp + u * G;
      if (c == 0 && r < t1) a.lse[r] = l[u];
    }
    const int bend = min(t1, b + U * G);
    while (t < bend) {
      if (end <= t) return;  // offsets that do not ascend
      const int to = min(bend, end);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = b + grp + u * G;
        if (b + u * G >= t1) break;
        if (!counted[u] || r < t || r >= to) continue;
#pragma unroll
        for (int i = 0; i < P * V; ++i) acc[i] = fmaf(rows[u].v[i], inv[u], acc[i]);
        if (ids[u] >= 0 && ids[u] < a.E) atomicAdd(&g.c[ids[u]], 1);
        for (int j = c + L; j < a.k; j += L) {
          const int32_t id = a.ids[(int64_t)r * a.k + j];
          if (id >= 0 && id < a.E) atomicAdd(&g.c[id], 1);
        }
        z = fmaf(l[u], l[u], z);
        ++n;
      }
      t = to;
      if (t != end && t != t1) continue;
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          g.p[grp][(q * L + c) * V + i] = acc[q * V + i];
          acc[q * V + i] = 0.f;
        }
      if (c == 0) {
        g.z[grp] = z;
        g.n[grp] = n;
      }
      z = 0.f;
      n = 0;
      lds_barrier();
      flush(s);
      if (t == t1) return;
      lds_barrier();
      for (int e = threadIdx.x; e < a.E; e += TH) g.c[e] = 0;
      s = seq_search(off, a.S, t);
      int lo;
      seq_rows(off, s, a.T, lo, end);
      lds_barrier();
    }
  }
}

// The rows of [t0, t1) that lie in sequences; the others' lse is written.
template <int TH>
__device__ __forceinline__ void clip_rows(const BalanceArgs& a, const Offsets& off, int& t0, int& t1) {
  if (!a.off) return;
  const int lo = min(max(off(0), 0), a.T), hi = min(max(off(a.S), 0), a.T);
  for (int t = t0 + threadIdx.x; t < t1; t += TH)
    if (t < lo || t >= hi) a.lse[t] = kNegInf;
  t0 = max(t0, lo);
  t1 = min(t1, hi);
}

template <int V, int L, int P>
__global__ __launch_bounds__(kThreadsB) void k_balance_rows(BalanceArgs a) {
  using Gt = Gathered<V, L, P, kThreadsB>;
  __shared__ Gt g;
  __shared__ int32_t lds[kSeqLds + 1];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.arrived = 0;
  const Offsets off = load_offsets<kThreadsB>(a.off, a.S, lds);
  int t0 = blockIdx.x * a.rows, t1 = min(a.T, t0 + a.rows);
  clip_rows<kThreadsB>(a, off, t0, t1);
  gather_rows<V, L, P, kThreadsB>(a, off, t0, t1, g, [&](int s) {
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
  });
}

// What the losses are made of: the terms of both, tokens, sequences with one
struct Sums {
  double balance, z;
  int32_t n, used;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.balance + y.balance, x.z + y.z, x.n + y.n, x.used + y.used};
}
// Sum over 16 neighbouring lanes, in each of them: by moves within the row of lanes, which
// cost an instruction each where a shuffle costs a hundred cycles
template <int CTRL> __device__ __forceinline__ double moved(double v) {
  return __hiloint2double(lane_move<CTRL>(__double2hiint(v)), lane_move<CTRL>(__double2loint(v)));
}
template <int CTRL> __device__ __forceinline__ Sums add_moved(const Sums& v) {
  return v + Sums{moved<CTRL>(v.balance), moved<CTRL>(v.z), lane_move<CTRL>(v.n), lane_move<CTRL>(v.used)};
}
__device__ __forceinline__ Sums sum16(Sums v) {
  v = add_moved<0xb1>(v);      // quad_perm 1,0,3,2
  v = add_moved<0x4e>(v);      // quad_perm 2,3,0,1
  v = add_moved<0x141>(v);     // row_half_mirror
  return add_moved<0x140>(v);  // row_mirror
}
// Sums over a workgroup's 1024 threads, in every thread; the order is fixed.  sh: one per
// wave, which nothing reads any more.
constexpr int kSumWaves = 16;
__device__ __forceinline__ Sums block_sum(Sums v, Sums* sh) {
  v = sum16(v);
#pragma unroll
  for (int d = 16; d < 64; d <<= 1)
    v = v + Sums{__shfl_xor(v.balance, d), __shfl_xor(v.z, d), __shfl_xor(v.n, d), __shfl_xor(v.used, d)};
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  lds_barrier();
  return sum16(sh[threadIdx.x & (kSumWaves - 1)]);
}
__device__ __forceinline__ void write_losses(const BalanceArgs& a, const Sums& s) {
  a.tokens[a.S] = s.n;
  a.tokens[a.S + 1] = s.used;
  a.loss[0] = (float)(s.used > 0 ? s.balance * a.E / s.used : 0.0);
  a.loss[1] = (float)(s.n > 0 ? s.z / s.n : 0.0);
}

// What workgroups leave for the last of them goes through the point that all dies share,
// value by value: a fence would write back and empty a die's whole cache, for each
// workgroup.
template <class T> __device__ __forceinline__ void give(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ T take(T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One workgroup of 1024 threads per COLS experts and sequence, the other lanes along the
// sequence's chunks.  All it does is wait: for the offsets, the
// slots, the others and what those left, each once.
static_assert(kFinishThreads == 64 * kSumWaves && kOneThreads == 64 * kSumWaves, "block_sum");
template <int COLS>
__global__ __launch_bounds__(kFinishThreads) void k_balance_finish(BalanceArgs a) {
  constexpr int CHUNKS = kFinishThreads / COLS;
  constexpr int W = kFinishThreads / 64;
  __shared__ double sp[W][COLS];
  __shared__ int32_t scn[W][COLS];
  __shared__ Sums sh[W];
  __shared__ int32_t last;
  const int nb = (a.E + COLS - 1) / COLS;
  const int s = blockIdx.x / nb, b = blockIdx.x % nb, w = threadIdx.x >> 6;
  const int col = threadIdx.x % COLS, ch = threadIdx.x / COLS, e = b * COLS + col;
  int lo, hi;
  seq_rows(Offsets{a.off, nullptr}, s, a.T, lo, hi);
  const int c0 = lo / a.rows, c1 = hi > lo ? (hi - 1) / a.rows + 1 : c0;
  double p = 0.0;
  int32_t cnt = 0;
  Sums mine = {};
  for (int c = c0 + threadIdx.x; c < c1; c += kFinishThreads) {
    mine.n += a.sum_n[c + s];
    mine.z += (double)a.sum_z[c + s];
  }
  if (e < a.E) {
#pragma unroll 8
    for (int c = c0 + ch; c < c1; c += CHUNKS) {
      const int64_t i = ((int64_t)c + s) * a.E + e;
      p += (double)a.sum_p[i];
      cnt += a.sum_c[i];
    }
  }
#pragma unroll
  for (int d = COLS; d < 64; d <<= 1) {
    p += __shfl_xor(p, d);
    cnt += __shfl_xor(cnt, d);
  }
  if ((threadIdx.x & 63) < COLS) {
    sp[w][col] = p;
    scn[w][col] = cnt;
  }
  const Sums all = block_sum(mine, sh);
  if (threadIdx.x < COLS) {
    p = sp[0][col];
    cnt = scn[0][col];
#pragma unroll
    for (int q = 1; q < W; ++q) {
      p += sp[q][col];
      cnt += scn[q][col];
    }
    double term = 0.0;
    if (e < a.E) {
      a.counts[(int64_t)s * a.E + e] = cnt;
      if (all.n > 0) term = (double)cnt * p / ((double)a.k * all.n * all.n);
    }
    term = sum16({term, 0.0, 0, 0}).balance;
#pragma unroll
    for (int d = 16; d < COLS; d <<= 1) term += __shfl_xor(term, d);
    if (threadIdx.x == 0) {
      if (b == 0) {
        give(&a.tokens[s], all.n);
        give(&a.part_z[s], all.z);
      }
      give(&a.part[blockIdx.x], term);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // they have arrived, then this counts
      last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  lds_barrier();
  if (!last) return;
  mine = {};
  for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x; i += kFinishThreads) mine.balance += take(&a.part[i]);
  for (int i = threadIdx.x; i < a.S; i += kFinishThreads) {
    const int32_t m = take(&a.tokens[i]);
    mine.z += take(&a.part_z[i]);
    mine.n += m;
    mine.used += m > 0;
  }
  mine = block_sum(mine, sh);
  if (threadIdx.x == 0) write_losses(a, mine);
}

// All of it in one workgroup, one sequence after the other
template <int V, int L, int P>
__global__ __launch_bounds__(kOneThreads) void k_balance_one(BalanceArgs a) {
  using Gt = Gathered<V, L, P, kOneThreads>;
  __shared__ Gt g;
  __shared__ Sums sh[kOneThreads / 64];
  __shared__ int32_t lds[kOneSeqs + 1];
  const Offsets off = load_offsets<kOneThreads>(a.off, a.S, lds);
  Sums total = {};
  int t0 = 0, t1 = a.T;
  clip_rows<kOneThreads>(a, off, t0, t1);
  gather_rows<V, L, P, kOneThreads>(a, off, t0, t1, g, [&](int s) {
    Sums v = {};
    if (threadIdx.x < Gt::GROUPS) {
      v.n = g.n[threadIdx.x];
      v.z = (double)g.z[threadIdx.x];
    }
    for (int e = threadIdx.x; e < a.E; e += kOneThreads) {
      const int32_t cnt = g.c[e];
      a.counts[(int64_t)s * a.E + e] = cnt;
      double p = 0.0;
#pragma unroll 8
      for (int q = 0; q < Gt::GROUPS; ++q) p += (double)g.p[q][e];
      v.balance += (double)cnt * p;
    }
    v = block_sum(v, sh);
    if (threadIdx.x == 0) {
      a.tokens[s] = v.n;
      if (v.n > 0) total = total + Sums{v.balance / ((double)a.k * v.n * v.n), v.z, v.n, 1};
    }
  });
  for (int s = 0; s < a.S; ++s) {  // without rows
    int lo, hi;
    seq_rows(off, s, a.T, lo, hi);
    if (lo < hi) continue;
    for (int e = threadIdx.x; e < a.E; e += kOneThreads) a.counts[(int64_t)s * a.E + e] = 0;
    if (threadIdx.x == 0) a.tokens[s] = 0;
  }
  if (threadIdx.x == 0) write_losses(a, total);
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

// A group of L lanes takes `per` consecutive rows, so that the f of their sequence
// stay in registers from row to row.  STREAM: the gradient and what is added to it
// bypass the caches' retention.
template <int V, int L, int P, bool STREAM>
__global__ __launch_bounds__(kThreadsB) void k_balance_grad(BalanceGradArgs a) {
  __shared__ int32_t lds[kSeqLds + 1];
  const int c = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const Offsets off = load_offsets<kThreadsB>(a.off, a.S, lds);
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
      const int s = !a.off ? 0 : seq >= 0 && t < off(seq + 1) ? seq : seq_search(off, a.S, t);
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
      float dot = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < P * V; ++i) {
        r.v[i] = expf(r.v[i] - l);
        dot = fmaf(f[i], r.v[i], dot);
        sum += r.v[i];
      }
      const float inv = __builtin_amdgcn_rcpf(group_reduce<L>(sum, Sum()));  // good to a step
      dot = group_reduce<L>(dot, Sum()) * inv;
      const float kp = ks * inv, kl = kz * inv;
      // (kl p first: kl lse may be past fp32's range where p is small, or 0)
#pragma unroll
      for (int i = 0; i < P * V; ++i)
        ad.v[i] = fmaf(kl * r.v[i], l, fmaf(kp * r.v[i], f[i] - dot, ad.v[i]));
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

bool matrix16(const float* p, int64_t ld, int32_t E) { return aligned(p, 16) && ld % 4 == 0 && E % 4 == 0; }
moe_status_t launched_b() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Gradients from this size on are stored past the caches.
constexpr int64_t kStreamGrad = 16 << 20;

}  // namespace

}  // namespace moe_mx

using namespace moe_mx;

extern "C" size_t moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t S) {
  if (!balance_sizes_valid(T, E, 1, S) || !balance_sizes_supported(T, E, 1, S)) return 0;
  return balance_plan(T, E, S).total;
}

extern "C" moe_status_t moe_balance(const float* logits, int64_t logits_ld, const int32_t* topk_ids,
                                    const uint8_t* mask, const int32_t* seq_offsets, int32_t T, int32_t E, int32_t k,
                                    int32_t S, float* loss, int32_t* counts, int32_t* tokens, float* lse,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!balance_sizes_valid(T, E, k, S) || (!seq_offsets && S != 1)) return MOE_ERR_INVALID_ARG;
  if (!balance_sizes_supported(T, E, k, S)) return MOE_ERR_UNSUPPORTED;
  if (!loss || !counts || !tokens || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(tokens, 4) ||
      !aligned(seq_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !lse || logits_ld < E || !aligned(logits, 4) || !aligned(topk_ids, 4) ||
                !aligned(lse, 4)))
    return MOE_ERR_INVALID_ARG;
  const BalancePlan f = balance_plan(T, E, S);
  if (f.total > 0 && (!workspace || workspace_bytes < f.total)) return MOE_ERR_WORKSPACE;
  if (f.total > 0 && !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
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
    for_row_shape<true>(vec, E, [&](auto V, auto L, auto P) {
      k_balance_one<V.value, L.value, P.value><<<1, kOneThreads, 0, stream>>>(a);
    });
    return launched_b();
  }
  char* ws = (char*)workspace;
  a.rows = f.rows;
  a.sum_p = (float*)(ws + f.sum_p);
  a.sum_c = (int32_t*)(ws + f.sum_c);
  a.sum_z = (float*)(ws + f.sum_z);
  a.sum_n = (int32_t*)(ws + f.sum_n);
  a.part = (double*)(ws + f.part);
  a.part_z = (double*)(ws + f.part_z);
  a.arrived = (uint32_t*)(ws + f.arrived);
  for_row_shape<true>(vec, E, [&](auto V, auto L, auto P) {
    k_balance_rows<V.value, L.value, P.value><<<(unsigned)std::max(f.chunks, 1), kThreadsB, 0, stream>>>(a);
  });
  const moe_status_t r = launched_b();
  if (r != MOE_OK) return r;
  const unsigned finish = (unsigned)S * (unsigned)f.blocks;
  if (f.cols == 64) k_balance_finish<64><<<finish, kFinishThreads, 0, stream>>>(a);
  else k_balance_finish<16><<<finish, kFinishThreads, 0, stream>>>(a);
  return launched_b();
}

extern "C" moe_status_t moe_balance_backward(const float* dloss, const float* logits, int64_t logits_ld,
                                             const int32_t* counts, const int32_t* tokens, const float* lse,
                                             const int32_t* seq_offsets, int32_t T, int32_t E, int32_t k, int32_t S,
                                             const float* add, int64_t add_ld, float* dlogits, int64_t dlogits_ld,
                                             hipStream_t stream) {
  if (!balance_sizes_valid(T, E, k, S) || (!seq_offsets && S != 1)) return MOE_ERR_INVALID_ARG;
  if (!balance_sizes_supported(T, E, k, S)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dloss || !logits || !counts || !tokens || !lse || !dlogits || logits_ld < E || dlogits_ld < E ||
      (add && add_ld < E))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {(const void*)dloss, (const void*)logits, (const void*)counts, (const void*)tokens,
                        (const void*)lse, (const void*)seq_offsets, (const void*)add, (const void*)dlogits})
    if (!aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  BalanceGradArgs a = {dloss, logits, logits_ld, counts, tokens, lse, seq_offsets, T, E, k, S, 1,
                       add,   add_ld, dlogits,   dlogits_ld};
  const bool vec = matrix16(logits, logits_ld, E) && matrix16(dlogits, dlogits_ld, E) &&
                   (!add || matrix16(add, add_ld, E));
  const bool stream_out = (int64_t)T * E * 4 >= kStreamGrad;
  for_row_shape<false>(vec, E, [&](auto V, auto L, auto P) {
    constexpr int G = kThreadsB / L.value;
    a.per = balance_grad_rows(T, G);
    const int64_t blocks = balance_grad_blocks(T, G);
    if (stream_out) k_balance_grad<V.value, L.value, P.value, true><<<(unsigned)blocks, kThreadsB, 0, stream>>>(a);
    else k_balance_grad<V.value, L.value, P.value, false><<<(unsigned)blocks, kThreadsB, 0, stream>>>(a);
  });
  return launched_b();
}
