// mx4_linear with many rows: tiles of 64 MSUB rows by 256 columns on the block-scaled
// MFMA v_mfma_scale_f32_32x32x64_f8f6f4 with E2M1 on both sides (mxfp6-sm120 page,
// "Execution model"; TokenSpeed SiTU page, "Supported contract": MxE2m1).
//
//   v[m, n] = sum_b 2^(sa[m, b] + sw[n, b] - 254) sum_{k in block b} a[m, k] w[n, k] + bias[n]
//   out[m, n] = bf16(fn(v) mul[m, n] + residual[m, n])
// The instruction applies both scales of a block of 32 to 64 k at a time and adds in fp32;
// accumulators stay in registers from the first k to the epilogue.
//
// Bound.  With E2M1 on both sides the instruction takes 32 cycles, half of E4M3's, and moves
// half the bytes, so that everything around it counts twice.  On values of any size registers
// alone reach 5.8 to 6.2 PFLOP/s (the clock gives way to power; zeros reach 9.7).  A wave that
// has its SIMD to itself pays for each instruction of its own beside its MFMAs, and that is what
// bounds a stage of 256 k: 2680 cycles with 256 rows for 2048 of MFMAs, 1820 with 128 rows for
// 1024, beside which it has 33 vector, 89 scalar, 29 LDS and 14 copy instructions, some 4.5
// cycles each (counters; 26 of the scalar ones set M0 for the copies).  LDS is busy for a quarter
// of the time, a quarter of that with conflicts.  Waits (first stages, epilogues, barriers) take
// a fifth of a wave's time, an item's epilogue and what stands around it 10600 cycles with 128
// rows.  What each choice is for:
// - Four waves, one per SIMD, of 32 MSUB x 128 each: the largest pieces of the accumulator, so
//   the fewest fragments (6 reads for 8 MFMAs with 128 rows, 8 for 16 with 256).  Eight waves
//   spill (8192^3: 316 us for 304); two workgroups a CU of 128 rows, 128 k a stage, to have one's
//   epilogue beside the other's products, fetch every scale line four times as often and rows
//   by 64 bytes (469 us for 319).
// - Stages of 256 k, rows of 128 bytes, a cache line; of 128 k: 279 us for 255 (256 rows).
// - Two slots of stages, three where they fit (64 and 128 rows).  Scales travel in groups of
//   two stages, 16 bytes a row; three slots of 128 rows leave room for two groups, which are
//   enough where every item has an even number of stages (8192^3: 319 us -> 310; 65536 rows of
//   128 experts, 1536 x 4096: 365 -> 338).
// - Copies go from memory to LDS without registers, a stage's spread between the MFMAs of two
//   steps; fragments are read a step ahead.  No branch stands among MFMAs: it would end the
//   block that the compiler can interleave.
// - Workgroups are persistent and walk patches of 4 row tiles by 8 column blocks per XCD, so
//   that 32 of them share what they read in its L2 (copies alone, 8192^3: 239 us -> 214).
// - The next item's copies are under way during an epilogue, and biases come with them: loaded
//   in the epilogue they wait for every copy before them (512 rows of 384 experts, 7168 x 2048:
//   474 us -> 377).
// - Few dense items of 64 rows split K into ranges, whose fp32 sums a second launch joins.
//
// Measured (MI355X, from codes): 8192 x 8192 x 8192 262 us with 256 rows, 4.2 PFLOP/s, 128 rows
// 310, 64 rows 415; 8192 x 4096 x 7168 119, 143, 183; 65536 rows of 128 experts, 1536 x 4096, 289,
// 310, 420 and, 128 rows, with SiLU 338, with a second factor 350, with both 376.  What is left:
// the instructions beside the MFMAs, epilogues that the next item's products do not overlap (about
// 5 us of a 128-row item's 21), the padding of a group's last tile, and a launch's last round.
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "copy_ring.h"
#include "epilogue.h"
#include "gemm.h"
#include "mx_device.h"

namespace moe_mx {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kThreads4 = 256;
constexpr int TN = kFp4Cols;
constexpr int ROW = 128;  // bytes of a row per stage: 256 K

template <int MSUB, int SLOTS_> struct Lay4 {
  static constexpr int TM = 64 * MSUB;
  static constexpr int NBUF = SLOTS_;
  static constexpr int SA = TM * ROW, SB = TN * ROW, STAGE = SA + SB;
  // Scales travel in groups of two stages, 16 bytes a row.  While a stage is begun, the groups
  // of the NBUF - 1 before it are in use: with three slots, of two groups if every item's
  // stages pair up, else of up to three (64 rows have room for four).
  static constexpr int GA = TM * 16, GROUP = GA + TN * 16;
  static constexpr int GBUFS = MSUB == 1 ? 4 : 2;
  static constexpr int SCALES = NBUF * STAGE;
  // Biases of the items that have a stage under way (K >= 512: two stages an item), 256
  // columns each.
  static constexpr int BIAS = SCALES + GBUFS * GROUP, BBUFS = 3;
  static constexpr int TOTAL = BIAS + BBUFS * 4 * TN;
  static constexpr int ACOP = TM / 32, BCOP = TN / 32;  // 1-KB copies per wave and stage
  static_assert(TOTAL <= 160 * 1024, "LDS");
};

struct Item4 {
  int expert, p0, rows, nb;
  int range, k0, kend;  // of the ranges of K; its stages
};
// The items of an XCD, q, q + Q, ... for its workgroup q: patches of kPatchM row tiles
// by kPatchN column blocks one after the other, so that workgroups that run at the
// same time share what they read in the XCD's L2.  Row tiles go to the XCDs in blocks
// of kPatchM; those behind the last 8 whole blocks are shared out item by item.
constexpr int kPatchM = 4, kPatchN = 8;
struct Sched4 {
  int xcd, full, tail0, q, Q, NB, ntiles, nk, items;
  int len;   // stages of a range of K
  bool odd;  // K % 256 == 128: the last stage is half of one
};

template <int TM, bool SPLIT>
__device__ __forceinline__ Item4 item_at(const FcArgs& p, const Sched4& sc, int li) {
  const int j = sc.q + li * sc.Q, block = kPatchM * sc.NB;
  int u, t0;  // item within a run of blocks that begins with tile t0
  if (j < sc.full * block) {
    u = j % block;
    t0 = kPatchM * (8 * (j / block) + sc.xcd);
  } else {
    u = sc.tail0 + j - sc.full * block;
    t0 = 8 * kPatchM * sc.full + kPatchM * (u / block);
    u %= block;
  }
  const int rows = min(kPatchM, sc.ntiles - t0), nb0 = u / (rows * kPatchN) * kPatchN;
  u -= rows * nb0;
  const int width = min(kPatchN, sc.NB - nb0), ti = __builtin_amdgcn_readfirstlane(t0 + u / width);
  Item4 it;
  it.nb = __builtin_amdgcn_readfirstlane(nb0 + u % width);
  it.range = it.k0 = 0;
  it.kend = sc.nk;
  if (SPLIT) {
    it.range = __builtin_amdgcn_readfirstlane(it.nb / p.nchunks);
    it.nb = __builtin_amdgcn_readfirstlane(it.nb - it.range * p.nchunks);
    it.k0 = it.range * sc.len;
    it.kend = min(sc.nk, it.k0 + sc.len);
  }
  if (p.dense_rows > 0) {
    it.expert = 0;
    it.p0 = TM * ti;
    it.rows = min(TM, p.dense_rows - TM * ti);
  } else {
    const Tile t = load_tile(p.tiles, ti);
    it.expert = t.expert;
    it.p0 = t.p0;
    it.rows = t.rows;
  }
  return it;
}

// A matrix for buffer loads: byte offsets from `base` below 2^31 are read, others give zeros.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ v4i buffer_of(const void* base) {
  const uint64_t a = (uint64_t)base;
  return (v4i){__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xffff), (int)kOutside, 0x00020000};
}
// Lane i's 16 bytes at off + soff of the buffer to LDS at lds + 16 i
__device__ __forceinline__ void lds_copy16_b(v4i buffer, uint32_t off, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)),
               "v"(off), "s"(buffer), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}

// The copies of one wave: stages in order, each in COPIES parts that the caller
// spreads between its MFMAs.
template <int MSUB, int NBUF, bool BIAS, bool SPLIT> struct Copier {
  using L = Lay4<MSUB, NBUF>;
  static constexpr int COPIES = L::ACOP + L::BCOP;
  const FcArgs& p;
  const Sched4& sc;
  uint32_t lds0;
  int w, lane;
  // cursor: items begun, stage of the last, LDS offsets of its stage and scale group
  int li = 0, ls, slot = 0, group = 0, bbuf = 0;
  int k0, kend;  // the stages of its item
  // the item and stage that parts belong to
  v4i abuf, wbuf;
  const uint8_t *asb, *wsb;
  uint32_t aoff[L::ACOP], boff[L::BCOP], asoff, wsoff, outside[2], soff, dst;
  int64_t bias_at;  // of the bias, in elements
  int cols;         // columns from the item's first one on

  // The block that copy i of this lane brings to its place of a row: block c of row r lies at
  // place c ^ (r >> 1 & 7), so that 16 rows read at the same block meet all of the banks.
  // (Rows 8 i + lane / 8; a wave's copies begin at an even i.)
  __device__ __forceinline__ int chunk(int i) const { return (lane & 7) ^ (lane >> 4 | (i & 1) << 2); }
  __device__ __forceinline__ void set_item() {
    const Item4 it = item_at<L::TM, SPLIT>(p, sc, li);
    const int K = p.K, kb = K / 2, ks = K / 32, n0 = it.nb * TN, last = p.N - 1 - n0;
    const int r8 = lane >> 3;
    abuf = buffer_of((const uint8_t*)p.a + (int64_t)it.p0 * kb);
    wbuf = buffer_of(p.w + (int64_t)it.expert * p.w_estride + (int64_t)n0 * kb);
    asb = p.a_scale + (int64_t)it.p0 * ks;
    wsb = p.w_scale + (int64_t)it.expert * p.ws_estride + (int64_t)n0 * ks;
#pragma unroll
    for (int i = 0; i < L::ACOP; ++i)
      aoff[i] = (uint32_t)min(8 * (L::ACOP * w + i) + r8, it.rows - 1) * (uint32_t)kb + 16 * chunk(i);
#pragma unroll
    for (int i = 0; i < L::BCOP; ++i)
      boff[i] = (uint32_t)min(epi_row32(8 * (L::BCOP * w + i) + r8), last) * (uint32_t)kb + 16 * chunk(i);
    asoff = (uint32_t)min(64 * min(w, MSUB - 1) + lane, it.rows - 1) * (uint32_t)ks;
    wsoff = (uint32_t)min(epi_row32(64 * w + lane), last) * (uint32_t)ks;
    bias_at = (int64_t)it.expert * p.N + n0;
    cols = last + 1;
    k0 = it.k0;
    kend = it.kend;
  }
  // Goes to the next stage.  Past the last stage of the last item that stage goes out
  // again, into a slot that nothing reads any more: without a branch around them the
  // copies can stand between the MFMAs.
  // (In four pieces, to stand between MFMAs: each is computed where it is called, not where
  // it is used.)
  __device__ __forceinline__ void advance(int piece) {
    if (piece == 0) {
      dst = lds0 + slot;
      asm volatile("" : "+s"(dst));
    } else if (piece == 1) {
      slot = slot == (L::NBUF - 1) * L::STAGE ? 0 : slot + L::STAGE;
      asm volatile("" : "+s"(slot));
    } else if (piece == 2) {
      ls = min(ls + 1, kend - 1);
      soff = ROW * ls;
      asm volatile("" : "+s"(ls), "+s"(soff));
    } else {
      // the half stage at the end of K: zeros for the second half
      const bool half = sc.odd && ls == sc.nk - 1;
      outside[0] = half && chunk(0) >= 4 ? kOutside : 0;
      outside[1] = half && chunk(1) >= 4 ? kOutside : 0;
      asm volatile("" : "+v"(outside[0]), "+v"(outside[1]));
    }
  }
  __device__ __forceinline__ bool ends_item() const { return ls == kend - 1 && li < sc.items; }
  __device__ __forceinline__ void next_item() {
    set_item();
    ++li;
    ls = k0 - 1;
  }
  __device__ __forceinline__ bool scales() const { return (ls & 1) == 0; }
  // the stage's scale group, where it is the first of two
  __device__ __forceinline__ void begin() {
    if (scales()) {
      const int s0 = min(8 * ls, p.K / 32 - 16);
      const uint32_t g = lds0 + L::SCALES + group;
      lds_copy16_s(asb + s0, asoff, g + 1024 * min(w, MSUB - 1));
      lds_copy16_s(wsb + s0, wsoff, g + L::GA + 1024 * w);
      group = group == (L::GBUFS - 1) * L::GROUP ? 0 : group + L::GROUP;
    }
    if (BIAS && ls == 0) bias();
  }
  // the item's bias as it is, a dword a lane; bf16 from the dword on that holds its first value
  __device__ __forceinline__ void bias() {
    const Epilogue e = epi_load();
    const bool f32 = e.bias_kind == kBiasF32 || e.bias_kind == kBiasF32Any;
    const uint64_t at = (uint64_t)e.bias + (f32 ? 4 : 2) * bias_at;
    const int last = f32 ? cols - 1 : (cols - 1 + ((int)at >> 1 & 1)) >> 1;
    lds_copy4_s((const uint8_t*)(at & ~(uint64_t)3), 4 * min(64 * w + lane, last), lds0 + L::BIAS + bbuf + 256 * w);
    bbuf = bbuf == (L::BBUFS - 1) * 4 * TN ? 0 : bbuf + 4 * TN;
  }
  __device__ __forceinline__ void part(int i) {
    if (i < L::ACOP) lds_copy16_b(abuf, aoff[i] | outside[i & 1], soff, dst + 1024 * (L::ACOP * w + i));
    else lds_copy16_b(wbuf, boff[i - L::ACOP] | outside[i & 1], soff, dst + L::SA + 1024 * (L::BCOP * w + i - L::ACOP));
  }
};

// f(0), f(1), ... with compile-time arguments
template <int N> using Int = std::integral_constant<int, N>;
template <class F, int... I>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(Int<I>()), ...);
}

// Epilogue of a wave, 32 rows by 64 columns at a time: part (h, m) holds row 32 (wm + 2m) + l32
// of the tile and in each lane four pieces of eight columns, at col + 64 h + 16 q.  IN: there
// is a second factor or a residual.
//
// A wave has its SIMD to itself, so this costs what its instructions cost, some 4.5 cycles
// each: 10000 of them (32 pieces one behind the other, each with its bounds, bias and
// function) took 47000 cycles an item, half of a K loop of 8192.  So the parts of a half run in
// a loop, with branches around what is absent; the accumulators are picked by a branch
// too, read by assembly, which the compiler cannot turn into selections over all of them.
// Stores count on the same in-order counter as loads and copies, and take microseconds
// while every workgroup writes.  Nothing here waits for one: loads go out a part ahead, and
// no branch stands around a store or a load, so that the compiler can count those behind the
// one it waits for (pieces outside the tile or N: an offset outside the buffer).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ float acc_read(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}
// silu of epilogue.h with the hardware's exponential: t is off by |v| + 2 half steps of fp32 for
// a few, which v t, at most 0.28, leaves below half a step of 1 in the result; for v below -87.3
// (results smaller than 1e-36) t may be 0.  (12 instructions for 30: 65536 rows of 128 experts,
// with a second factor, took 446 us with it and 392 with this.)
__device__ __forceinline__ void fn_of(int fn, float (&v)[8]) {
  if (fn == MX_FN_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __builtin_amdgcn_exp2f(fabsf(v[i]) * -1.44269504f);
      v[i] = v[i] * (v[i] < 0.0f ? t : 1.0f) * __builtin_amdgcn_rcpf(1.0f + t);
    }
  } else {
    epi_fn(fn, v);
  }
}

template <int MSUB, bool IN, bool BIAS>
__device__ __forceinline__ void finish(v16f (&acc)[MSUB][4], const Item4& it, int N, int wm, int l32, int col,
                                       const uint8_t* biases) {
  // the last MFMAs' results, for the assembly below
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  const Epilogue e = epi_load();
  const int64_t tile = (int64_t)it.p0 * N;
  auto buffer = [&](const void* q) {
    return __builtin_amdgcn_make_buffer_rsrc(q ? (uint16_t*)q + tile : nullptr, 0, q ? (int)kOutside : 0, 0x00020000);
  };
  const auto out = buffer(e.out), mul = buffer(e.mul), res = buffer(e.residual);
  const bool has_mul = e.mul != nullptr;
  const int rows = it.rows - 32 * wm - l32, cols = N - col;  // of this lane's first row and column on
  const int first = (int)(2 * ((uint32_t)(32 * wm + l32) * (uint32_t)N + col));
  auto at = [&](int h, int m, int q) {
    const int side = 64 * h + 16 * q < cols ? 0 : (int)kOutside;
    return ((64 * m < rows ? first + 128 * h + m * (128 * N) : (int)kOutside) | side) + 32 * q;
  };
  // what a part takes in goes out AHEAD parts before it: all of it with up to 128 rows, whose
  // registers have room, two with 256 (8192^3 with a residual: one 314 us, two 296)
  constexpr int AHEAD = MSUB <= 2 ? 2 * MSUB : 2;
  u32x4 nm[AHEAD][4], nr[AHEAD][4];
  auto request = [&](int slot, int h, int m) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      nm[slot][q] = __builtin_amdgcn_raw_buffer_load_b128(mul, at(h, m, q), 0, 0);
      nr[slot][q] = __builtin_amdgcn_raw_buffer_load_b128(res, at(h, m, q), 0, 0);
    }
  };
  if constexpr (IN) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) request(j, j / MSUB, j % MSUB);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    auto part = [&](int m, int slot) {
      float v[4][8];
      each(std::make_integer_sequence<int, MSUB>(), [&](auto M) {
        if (m == M.value) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[q][i] = acc_read(acc[M.value][2 * h + (i >> 2)][4 * q + (i & 3)]);
        }
      });
      if constexpr (BIAS) {
        const int c = col % TN + 64 * h;
        if (e.bias_kind == kBiasF32 || e.bias_kind == kBiasF32Any) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float b[8];
            *(float4*)b = *(const float4*)(biases + 4 * (c + 16 * q));
            *(float4*)(b + 4) = *(const float4*)(biases + 4 * (c + 16 * q) + 16);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q][i] += b[i];
          }
        } else if (e.bias_kind == kBiasBf16) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 x = *(const uint4*)(biases + 2 * (c + 16 * q));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[q][i] += __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
          }
        } else {
          const uint8_t* first = biases + ((uint64_t)e.bias & 2);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[q][i] += __uint_as_float((uint32_t) * (const uint16_t*)(first + 2 * (c + 16 * q + i)) << 16);
        }
      }
      if (e.fn != MX_FN_NONE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) fn_of(e.fn, v[q]);
      }
      if constexpr (IN) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x = nm[slot][q][i / 2], y = nr[slot][q][i / 2];
            v[q][i] *= has_mul ? __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16) : 1.0f;
            v[q][i] += __uint_as_float(i & 1 ? y & 0xffff0000u : y << 16);
          }
        // (h, m) two parts on; behind the last one, that one again
        if constexpr (MSUB > AHEAD) {
          const int next = m + AHEAD < MSUB ? m + AHEAD : h ? MSUB - 1 : m + AHEAD - MSUB;
          request(slot, m + AHEAD < MSUB ? h : 1, next);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v2bf o2 = {(__bf16)v[q][2 * i], (__bf16)v[q][2 * i + 1]};
          uint32_t w;
          __builtin_memcpy(&w, &o2, 4);
          o[i] = w;
        }
        __builtin_amdgcn_raw_buffer_store_b128(o, out, at(h, m, q), 0, 0);
      }
    };
    if constexpr (MSUB <= 2) {
#pragma unroll
      for (int m = 0; m < MSUB; ++m) part(m, h * MSUB + m);
    } else {
#pragma unroll 1
      for (int m = 0; m < MSUB; m += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) part(m + j, j);
      }
    }
  }
}

// A range's sums in fp32, for launch_linear_join: 16 MSUB stores of every lane
template <int MSUB>
__device__ __forceinline__ void leave(v16f (&acc)[MSUB][4], const FcArgs& p, const Item4& it, int wm, int l32, int col) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  const auto out = __builtin_amdgcn_make_buffer_rsrc(p.part + ((int64_t)it.range * p.dense_rows + it.p0) * p.N, 0,
                                                     (int)kOutside, 0x00020000);
  const int rows = it.rows - 32 * wm - l32, cols = p.N - col;
#pragma unroll
  for (int m = 0; m < MSUB; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int h = j >> 2, q = j & 3;
      const bool in = 64 * m < rows && 16 * j < cols;
      const uint32_t at = in ? 4 * ((uint32_t)(32 * wm + l32 + 64 * m) * (uint32_t)p.N + col + 16 * j) : kOutside;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(acc_read(acc[m][2 * h + k][4 * q + i]));
        __builtin_amdgcn_raw_buffer_store_b128(o, out, (int)(at + 16 * k), 0, 0);
      }
    }
}

template <int MSUB, int NBUF, bool IN, bool BIAS, bool SPLIT>
__global__ __launch_bounds__(kThreads4, 1) void k_linear_fp4(FcArgs p) {
  using L = Lay4<MSUB, NBUF>;
  using C = Copier<MSUB, NBUF, BIAS, SPLIT>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[L::TOTAL];
  Sched4 sc;
  sc.nk = (p.K + 255) / 256;
  sc.odd = p.K % 256 != 0;
  const int ranges = SPLIT ? p.ksplit : 1;
  sc.len = SPLIT ? fp4_range(sc.nk, ranges) : sc.nk;
  sc.NB = p.nchunks * ranges;  // (ranges count as column blocks)
  sc.ntiles = p.dense_rows > 0 ? (p.dense_rows + L::TM - 1) / L::TM : *p.num_tiles;
  sc.xcd = blockIdx.x & 7;
  sc.q = blockIdx.x >> 3;
  sc.Q = gridDim.x >> 3;
  sc.full = sc.ntiles / (8 * kPatchM);
  const int tail = sc.ntiles % (8 * kPatchM) * sc.NB;
  sc.tail0 = tail * sc.xcd / 8;
  const int nitems = sc.full * kPatchM * sc.NB + tail * (sc.xcd + 1) / 8 - sc.tail0;
  sc.items = nitems > sc.q ? (nitems - sc.q + sc.Q - 1) / sc.Q : 0;
  if (sc.items == 0) return;

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1, l32 = lane & 31, g = lane >> 5;
  C copy{p, sc, lds_addr(smem), w, lane};

  // offsets of this lane's fragment of step s: row l32, block 4g + s at its place (Copier::chunk)
  int off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = l32 * ROW + 16 * ((4 * g + s) ^ (l32 >> 1 & 7));

  // fragments of two steps and scales of two stages: those in use and the next
  v4i fa[2][MSUB], fb[2][4];
  uint32_t sa[MSUB], sb[4], ta[MSUB], tb[4];
  v16f acc[MSUB][4];
  constexpr int READS = 4 + MSUB, SLOTS = 4 * MSUB;
  // fragment i of a step (offset o) of the stage at st
  auto read = [&](int f, const uint8_t* st, int o, int i) {
    if (i < 4) fb[f][i] = *(const v4i*)(st + L::SA + (4 * wn + i) * (32 * ROW) + o);
    else fa[f][i - 4] = *(const v4i*)(st + (wm + 2 * (i - 4)) * (32 * ROW) + o);
  };
  // scales of fragment i of the stage whose scales lie at gs
  auto read_scale = [&](const uint8_t* gs, int i) {
    if (i < 4) tb[i] = *(const uint32_t*)(gs + L::GA + 512 * (4 * wn + i));
    else ta[i - 4] = *(const uint32_t*)(gs + 512 * (wm + 2 * (i - 4)));
  };
  int cgroup = (L::GBUFS - 1) * L::GROUP;  // LDS offset of the scale group of the stage last read
  auto scales_at = [&](int ks) {
    if ((ks & 1) == 0) cgroup = cgroup == (L::GBUFS - 1) * L::GROUP ? 0 : cgroup + L::GROUP;
    const bool h = sc.odd && ks == sc.nk - 1;
    const int so = 8 * ks - min(8 * (ks & ~1), p.K / 32 - 16);
    return (uint32_t)(L::SCALES + cgroup + so + (16 * l32 + (h ? 0 : 4 * g)));
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int m = 0; m < MSUB; ++m) sa[m] = ta[m];
#pragma unroll
    for (int n = 0; n < 4; ++n) sb[n] = tb[n];
  };
  // The branches of copy.begin() end a basic block; without this the compiler moves the
  // MFMAs before it, whose results are only used after it, behind it and each other.
  auto pin = [&]() {
#pragma unroll
    for (int m = 0; m < MSUB; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) asm volatile("" : "+a"(acc[m][n]));
  };
  // MFMA k of step S on fragment set F
  auto mfma = [&](auto F, auto S, auto K) {
    constexpr int f = F.value, m = K.value / 4, n = K.value % 4, s = S.value;
    const v8i av = {fa[f][m][0], fa[f][m][1], fa[f][m][2], fa[f][m][3], 0, 0, 0, 0};
    const v8i bv = {fb[f][n][0], fb[f][n][1], fb[f][n][2], fb[f][n][3], 0, 0, 0, 0};
    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bv, av, acc[m][n], 4, 4, s, (int)sb[n], s, (int)sa[m]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // those of N operations f that come after MFMA K when they are spread over MFMAs [K0, K1)
  auto among = [&](auto K, auto N, auto K0, auto K1, auto f) {
    constexpr int n = N.value, k0 = K0.value, span = K1.value - K0.value;
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (k0 + i * span / n == K.value) f(i);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::make_integer_sequence<int, SLOTS> slots;
  constexpr Int<0> i0;
  constexpr Int<1> i1;
  constexpr Int<2> i2;
  constexpr Int<3> i3;
  constexpr Int<4> i4;
  constexpr Int<READS> reads;
  constexpr Int<C::COPIES / 2> half;
  constexpr Int<C::COPIES - C::COPIES / 2> rest;
  constexpr Int<SLOTS / 2> mid;
  constexpr Int<SLOTS * 3 / 4> late;
  constexpr Int<SLOTS> end;

  copy.next_item();
  const int first = copy.k0;
  for (int s = 0; s < L::NBUF; ++s) {
    if (copy.ends_item()) copy.next_item();
#pragma unroll
    for (int i = 0; i < 4; ++i) copy.advance(i);
    copy.begin();
#pragma unroll
    for (int i = 0; i < C::COPIES; ++i) copy.part(i);
  }
  wait_vm_lgkm0<0>();
  barrier();
  {
    const uint8_t* gs = smem + scales_at(first);
#pragma unroll
    for (int i = 0; i < READS; ++i) {
      read_scale(gs, i);
      read(0, smem, off[0], i);
    }
  }
  take_scales();
  const uint8_t* st = smem;
  int slot = 0, bbuf = 0;
  for (int ci = 0; ci < sc.items; ++ci) {
    const Item4 it = item_at<L::TM, SPLIT>(p, sc, ci);
#pragma unroll
    for (int m = 0; m < MSUB; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
    for (int ks = it.k0; ks < it.kend; ++ks) {
      each(slots, [&](auto k) {
        mfma(i0, i0, k);
        among(k, reads, i0, mid, [&](int i) { read(1, st, off[1], i); });
        among(k, rest, i0, end, [&](int i) { copy.part(half + i); });
      });
      each(slots, [&](auto k) {
        mfma(i1, i1, k);
        among(k, reads, i0, mid, [&](int i) { read(0, st, off[2], i); });
      });
      pin();
      const bool behind = copy.scales(), first = copy.ls == 0;  // (of the stage begun last)
      if (copy.ends_item()) copy.next_item();
      // (a range has more stages than the copies are ahead: they are in the next item)
      const int kn = ks + 1 < it.kend ? ks + 1 : SPLIT ? copy.k0 : 0;
      uint32_t so = 0;
      __builtin_amdgcn_sched_barrier(0);
      each(slots, [&](auto k) {
        mfma(i0, i2, k);
        among(k, reads, i0, mid, [&](int i) { read(1, st, off[3], i); });
        // the next stage's places
        among(k, i4, i0, end, [&](int i) { copy.advance(i); });
        if constexpr (k.value == SLOTS / 2) {
          slot = slot == (L::NBUF - 1) * L::STAGE ? 0 : slot + L::STAGE;
          asm volatile("" : "+s"(slot));
          __builtin_amdgcn_sched_barrier(0);
        } else if constexpr (k.value == SLOTS - 1) {
          so = scales_at(kn);
          asm volatile("" : "+v"(so));
          __builtin_amdgcn_sched_barrier(0);
        }
      });
      const uint8_t* gs = smem + so;
      pin();
      // every read of the stage has landed in this wave; the next stage has landed as a
      // whole once every wave passes the barrier, and this one's slot is free
      // (behind the copies of the item's first stages the epilogue before it has left 8
      // MSUB stores, and the first stage has sent the second half of the last once more)
      constexpr int kBehind = (SPLIT ? 16 : 8) * MSUB + rest;
      const bool stored = ks == it.k0 && ci > 0;
      if (L::NBUF == 2) {
        if (stored) wait_vm_lgkm0<kBehind>();
        else wait_vm_lgkm0<0>();
      } else if (BIAS && first) {  // and the stage after the next, begun last, is on its way
        if (stored) wait_vm_lgkm0<kBehind + C::COPIES + 3>();
        else wait_vm_lgkm0<C::COPIES + 3>();
      } else if (behind) {
        if (stored) wait_vm_lgkm0<kBehind + C::COPIES + 2>();
        else wait_vm_lgkm0<C::COPIES + 2>();
      } else {
        if (stored) wait_vm_lgkm0<kBehind + C::COPIES>();
        else wait_vm_lgkm0<C::COPIES>();
      }
      barrier();
      st = smem + slot;
      copy.begin();
      __builtin_amdgcn_sched_barrier(0);
      each(slots, [&](auto k) {
        mfma(i1, i3, k);
        among(k, reads, i0, mid, [&](int i) { read(0, st, off[0], i); });
        among(k, reads, i1, late, [&](int i) { read_scale(gs, i); });
        among(k, half, i0, end, [&](int i) { copy.part(i); });
      });
      take_scales();
      pin();
    }
    // The rest of the begun stage goes out before the stores, which the wait for it then need
    // not cover (the next item's first step sends it again: the same bytes, into a slot that is
    // not begun again before a wait for all of them).
#pragma unroll
    for (int i = half; i < C::COPIES; ++i) copy.part(i);
    // the lane holds row 32 (wm + 2m) + l32 of the tile, eight columns of each piece
    if constexpr (SPLIT) leave<MSUB>(acc, p, it, wm, l32, it.nb * TN + 128 * wn + 8 * g);
    else finish<MSUB, IN, BIAS>(acc, it, p.N, wm, l32, it.nb * TN + 128 * wn + 8 * g, smem + L::BIAS + bbuf);
    bbuf = bbuf == (L::BBUFS - 1) * 4 * TN ? 0 : bbuf + 4 * TN;
  }
  wait_vm_lgkm0<0>();  // no copy may land in LDS that is no longer this workgroup's
}

}  // namespace

template <int MSUB, int NBUF>
static void launch_fp4_t(const FcArgs& p, int grid, hipStream_t st) {
  const bool in = p.epi.mul || p.epi.residual, bias = p.epi.bias_kind != kBiasNone;
  auto kernel = in ? (bias ? k_linear_fp4<MSUB, NBUF, true, true, false> : k_linear_fp4<MSUB, NBUF, true, false, false>)
                   : (bias ? k_linear_fp4<MSUB, NBUF, false, true, false> : k_linear_fp4<MSUB, NBUF, false, false, false>);
  kernel<<<grid, kThreads4, 0, st>>>(p);
}

hipError_t launch_linear_fp4(const FcArgs& p, int rows, int grid, hipStream_t st) {
  if (grid < 8) grid = 8;
  grid &= ~7;
  if (p.ksplit > 1) {
    if (rows != 64 || p.dense_rows <= 0 || !fp4_range_ok((p.K + 255) / 256, p.ksplit)) return hipErrorInvalidValue;
    k_linear_fp4<1, 3, false, false, true><<<grid, kThreads4, 0, st>>>(p);
    return hipGetLastError();
  }
  const bool pairs = (p.K + 255) / 256 % 2 == 0;  // (Lay4: three slots of 128 rows)
  if (rows == 256) launch_fp4_t<4, 2>(p, grid, st);
  else if (rows == 128 && pairs) launch_fp4_t<2, 3>(p, grid, st);
  else if (rows == 128) launch_fp4_t<2, 2>(p, grid, st);
  else if (rows == 64) launch_fp4_t<1, 3>(p, grid, st);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace moe_mx
