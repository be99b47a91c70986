// mx_linear for few rows per weight matrix (a decode batch, or an expert's share
// of one), and for any K that is a multiple of 128: tiles of 16 or 64 rows, weights
// streamed through LDS.
//
// The bound is reading the packed weights from HBM once.  Loads straight into the
// MFMA layout touch one weight row per lane, 64 lines an instruction, and reach
// about half of the bandwidth; copies into LDS with eight neighbouring lanes on
// 128 (E2M1) or twelve on 192 (E3M2) contiguous bytes of a row keep HBM busy.  So
// one workgroup per CU runs seven waves (eight with 64 rows): 0-3 multiply, 4-5
// copy weights, the rest copy activations, over a ring of stages of 256 K, all but
// one of them in flight: 96 to 120 KB with 16 rows; with 64 rows 96 (E2M1), 80 (E3M2 x
// MXFP8), 56 (E3M2 x bf16: two stages).  A copy wave's memory counter drains in
// order, so before each stage's barrier it waits until only the copies of later
// stages remain.  Its addresses are a scalar base per stage and a 32-bit offset per
// lane that lasts for an item (64-bit ones per lane: 64-row tiles 3 to 8% slower).
//
// Measured (MI355X): 512 rows over 384 experts (64 tokens with 8 each; 283 experts
// have rows), N = 7168, K = 2048, 16-row tiles, with the rate of the weights' bytes:
//   E2M1 x bf16 416 us (5.3 TB/s), E2M1 x MXFP8 394 (5.6), E3M2 x bf16 557 (5.8),
//   E3M2 x MXFP8 553 (5.9); a copy of 1 GiB runs at 5.1.
// One matrix, N = 4096, K = 7168, in the same order: 64 rows in two K ranges of
// 16-row tiles 16.1, 16.6, 18.9, 18.6 us, in four of 64-row tiles 16.5, 17.0, 17.3,
// 18.1; 1024 rows in 64-row tiles 75, 54, 81, 66.  The weights of a dense matrix
// come from the caches; there the multiply waves' own instructions between two
// barriers bound it.  Eight multiply waves (4% slower), fragments of the next stage
// kept in registers ahead of time (E2M1 x MXFP8 4% faster, the others 4 to 18%
// slower) and wave priorities (no change) did not help.
//
// Work item = (row tile, 128 columns, K range); the persistent grid walks the
// items.  K may end in half a stage (K % 256 == 128): its copies repeat the first
// half and the second half is not multiplied.  Scales (8 bytes per row and stage)
// travel in groups of 4 stages of an item, 32 bytes per row in two 16-byte copies;
// one that would run past its row's end is moved back to end there.  Where a row
// has fewer than 16 bytes of them (SHORT: K < 512, one group per item) they are
// copied as words, 16 bytes per row, the last word again in place of those missing.
//
// Multiplication (lane = 16 g + r): each 128-K half of a stage is one MX block per
// lane of row r of a column tile, block g, against the same block of activation
// row r.  bf16 activations: weights are dequantized in registers (exact for E8M0
// scales) for four v_mfma_f32_16x16x32_bf16; MXFP8: one block-scaled MFMA.  The
// weights are the first operand and their rows are placed for epilogue.h.
#include <hip/hip_runtime.h>

#include "copy_ring.h"
#include "epilogue.h"
#include "gemm.h"
#include "mx_device.h"

namespace moe_mx {

namespace {

typedef int v6i __attribute__((ext_vector_type(6)));
typedef __bf16 v32bf __attribute__((ext_vector_type(32)));

constexpr int RN = kRowsCols;    // columns per item
// E3M2 weight row jr holds piece c of its 12 at slot (c + turn(jr)) % 12, so that the
// rows of a read, four of which would start at the same bank, are spread over them
__device__ __forceinline__ int turn(int jr) { return (jr >> 2) & 3; }
constexpr int RK = kRowsK;       // K per stage
constexpr int kMulWaves = 4, kWaveA = 6;
// activation-copy waves and threads for tiles of `sub` 16-row sub-tiles
constexpr int rows_awaves(int sub) { return sub == 1 ? 1 : 2; }
constexpr int rows_threads(int sub) { return 64 * (kWaveA + rows_awaves(sub)); }
constexpr int kGroupStages = 4;  // stages per scale group

// LDS: [stages: weights | activations] [weight scales] [activation scales]
// for tiles of SUB 16-row sub-tiles
template <bool MXA, int WF, int SUB, bool SHORT> struct Lay {
  static constexpr int RM = 16 * SUB;
  static constexpr int AWAVES = rows_awaves(SUB);
  static constexpr int BROW = RK * Fmt<WF>::BITS / 8;  // weight bytes per row and stage
  static constexpr int AROW = MXA ? RK : 2 * RK;       // activation bytes per row and stage
  static constexpr int S_B = RN * BROW, S_A = RM * AROW, STAGE = S_B + S_A;
  // as many stages as fit
  static constexpr int NST = STAGE <= 24 * 1024 ? 6 : STAGE <= 28 * 1024 ? 5 : STAGE <= 34 * 1024 ? 4
                             : STAGE <= 48 * 1024 ? 3 : 2;
  static constexpr int BCOP = S_B / 1024 / 2;          // 1-KB copies per weight wave and stage
  static constexpr int ACOP = S_A / 1024 / AWAVES;     // per activation wave and stage
  // Scales: bytes per row and group, group buffers, copies of a group per wave.  A
  // group is copied with its first stage x, after barrier x - NST + 1, which
  // certifies that stages up to x - NST are done with: the stages of the groups that
  // use the other buffers before it have to number NST - 1 <= 5 at least.  Items of
  // K >= 512 have two or more stages, so three neighbouring groups have (1, 4, 1 or
  // 2, 2, 2 at the least); SHORT ones have one at least.
  static constexpr int GROW = SHORT ? 16 : kGroupStages * RK / 32;
  static constexpr int BUFS = SHORT ? 8 : 4;
  static constexpr int WGCOP = SHORT ? 4 : 2;
  static constexpr int AGCOP = !SHORT || SUB == 1 ? 1 : 2;
  static constexpr int WS = NST * STAGE;               // weight scales
  static constexpr int WSB = RN * GROW;                // one buffer of them
  static constexpr int AS = WS + BUFS * WSB;           // activation scales
  static constexpr int ASB = (SHORT ? 256 : 1024) * AGCOP * AWAVES;  // one buffer
  static constexpr int TOTAL = AS + (MXA ? BUFS * ASB : 0);
  // copies that may be in flight when a stage is waited for
  template <int COP, int GCOP>
  static constexpr int IN_FLIGHT = (NST - 2) * COP + (SHORT ? NST - 2 : 2) * GCOP;
  static_assert(TOTAL <= 160 * 1024 && NST <= 6 && ASB >= RM * GROW, "LDS");
};

struct Item {
  int expert, p0, rows, nb, s0, ns;  // stages [s0, s0 + ns) of K
};
// NB column blocks and S ranges of the K stages per tile
struct Sched {
  int q, Q, NB, S, stages, items, total;
};

__device__ __forceinline__ int range0(const Sched& sc, int ks) { return ks * sc.stages / sc.S; }

template <int RM>
__device__ __forceinline__ Item item_at(const FcArgs& p, const Sched& sc, int li) {
  const int j = sc.q + li * sc.Q;
  const int ti = j / (sc.NB * sc.S), r = j % (sc.NB * sc.S);
  Item it;
  it.nb = r / sc.S;
  it.s0 = range0(sc, r % sc.S);
  it.ns = range0(sc, r % sc.S + 1) - it.s0;
  if (p.dense_rows > 0) {
    it.expert = 0;
    it.p0 = RM * ti;
    it.rows = min(RM, p.dense_rows - RM * ti);
  } else {
    const Tile t = load_tile(p.tiles, ti);
    it.expert = t.expert;
    it.p0 = t.p0;
    it.rows = t.rows;
  }
  return it;
}

// Half h (16 bytes, two stages) of the scale group that starts with stage s: its
// place in the row, moved back where the row ends before it does
__device__ __forceinline__ int scale_at(int s, int h, int row_bytes) { return min(8 * s + 16 * h, row_bytes - 16); }

// s_waitcnt vmcnt(n) lgkmcnt(0), n a run-time value in [LO, HI] (above HI: HI)
template <int LO, int HI>
__device__ __forceinline__ void wait_upto(int n) {
  if constexpr (LO == HI) {
    wait_vm_lgkm0<LO>();
  } else {
    constexpr int MID = (LO + HI + 1) / 2;
    if (n >= MID) wait_upto<MID, HI>(n);
    else wait_upto<LO, MID - 1>(n);
  }
}

// Order of a copy wave: issue(stage) makes COP copies, and GCOP of scales before
// them where the stage begins a scale group (it returns whether).  A stage has
// landed once at most the copies of the stages issued after it remain.
template <int NST, int COP, int GCOP, int IN_FLIGHT, class Issue>
__device__ __forceinline__ void copy_loop(const Sched& sc, Issue issue) {
  uint32_t hist = 0;  // bit i: the stage issued i before the last began a scale group
  int issued = 0;
  auto next = [&]() {
    hist = hist << 1 | (uint32_t)issue(issued);
    ++issued;
  };
  for (int s = 0; s < NST - 1 && s < sc.total; ++s) next();
  for (int g = 0; g < sc.total; ++g) {
    const int after = issued - 1 - g;
    wait_upto<0, IN_FLIGHT>(after * COP + GCOP * __popc(hist & ((1u << after) - 1u)));
    barrier();
    if (issued < sc.total) next();
  }
}

template <bool MXA, int WF, int SUB, bool SHORT>
__device__ __forceinline__ void copy_weights(const FcArgs& p, const Sched& sc, uint8_t* smem, int bw) {
  using L = Lay<MXA, WF, SUB, SHORT>;
  const int lane = threadIdx.x & 63;
  const uint32_t lds0 = lds_addr(smem);
  const int64_t wrow = (int64_t)p.K * Fmt<WF>::BITS / 8;
  const int srow = p.K / 32;
  const bool half = p.K % RK != 0;
  constexpr int CPR = L::BROW / 16;  // 16-byte pieces per row and stage
  // per lane, offsets from the item's first weight row (127 rows of K <= kMaxK values
  // of 3/4 byte fit 31 bits; so do 63 activation rows)
  const uint8_t* wb = nullptr;
  const uint8_t* sb = nullptr;
  uint32_t off[L::BCOP], soff[L::WGCOP];
  uint32_t back = 0;  // bit i: piece i of this lane lies in a stage's second half
  Item it = {};
  int li = 0, ls = 0, group = -1;
  auto issue = [&](int g) {
    if (ls == 0) {
      it = item_at<L::RM>(p, sc, li);
      const int n0 = it.nb * RN, last = p.N - 1 - n0;  // rows past N: the last one, not stored
      wb = p.w + (int64_t)it.expert * p.w_estride + n0 * wrow;
      sb = p.w_scale + (int64_t)it.expert * p.ws_estride + (int64_t)n0 * srow;
      back = 0;
#pragma unroll
      for (int i = 0; i < L::BCOP; ++i) {
        const int cc = 64 * (L::BCOP * bw + i) + lane, jr = cc / CPR;
        // E2M1: piece c of row jr at slot c ^ (jr & 7); E3M2: see turn()
        const int ch = WF == 1 ? (cc % CPR) ^ (jr & 7) : (cc % CPR + CPR - turn(jr)) % CPR;
        off[i] = (uint32_t)min(epi_row16(jr), last) * (uint32_t)wrow + 16 * ch;
        back |= (uint32_t)(ch >= CPR / 2) << i;
      }
#pragma unroll
      for (int i = 0; i < L::WGCOP; ++i) {
        const int jr = SHORT ? 64 * bw + 16 * i + (lane >> 2) : 64 * bw + 32 * i + (lane >> 1);
        soff[i] = (uint32_t)min(epi_row16(jr), last) * (uint32_t)srow;
      }
    }
    const int s = it.s0 + ls;
    const bool fresh = ls % kGroupStages == 0;
    if (fresh) {
      ++group;
      const uint32_t buf = lds0 + L::WS + (group % L::BUFS) * L::WSB;
#pragma unroll
      for (int i = 0; i < L::WGCOP; ++i) {
        if (SHORT) lds_copy4(sb + soff[i] + min(4 * (lane & 3), srow - 4), buf + 256 * (L::WGCOP * bw + i));
        else lds_copy16_s(sb, soff[i] + (uint32_t)scale_at(s, lane & 1, srow), buf + 1024 * (L::WGCOP * bw + i));
      }
    }
    const uint32_t base = lds0 + (g % L::NST) * L::STAGE;
    const uint8_t* ws = wb + (int64_t)s * L::BROW;
    if (half && s == sc.stages - 1) {
#pragma unroll
      for (int i = 0; i < L::BCOP; ++i)
        lds_copy16_s(ws, off[i] - (back >> i & 1 ? L::BROW / 2 : 0), base + 1024 * (L::BCOP * bw + i));
    } else {
#pragma unroll
      for (int i = 0; i < L::BCOP; ++i) lds_copy16_s(ws, off[i], base + 1024 * (L::BCOP * bw + i));
    }
    if (++ls == it.ns) {
      ls = 0;
      ++li;
    }
    return fresh;
  };
  copy_loop<L::NST, L::BCOP, L::WGCOP, L::template IN_FLIGHT<L::BCOP, L::WGCOP>>(sc, issue);
}

template <bool MXA, int WF, int SUB, bool SHORT>
__device__ __forceinline__ void copy_rows(const FcArgs& p, const Sched& sc, uint8_t* smem, int aw) {
  using L = Lay<MXA, WF, SUB, SHORT>;
  const int lane = threadIdx.x & 63;
  const uint32_t lds0 = lds_addr(smem);
  const bool half = p.K % RK != 0;
  const int64_t arow = MXA ? p.K : 2 * (int64_t)p.K;
  const int srow = p.K / 32;
  constexpr int CPR = L::AROW / 16;
  const uint8_t* ab = nullptr;
  const uint8_t* sb = nullptr;
  uint32_t off[L::ACOP], soff[L::AGCOP] = {};
  uint32_t back = 0;
  Item it = {};
  int li = 0, ls = 0, group = -1;
  auto issue = [&](int g) {
    if (ls == 0) {
      it = item_at<L::RM>(p, sc, li);
      ab = (const uint8_t*)p.a + it.p0 * arow;
      if (MXA) sb = p.a_scale + (int64_t)it.p0 * srow;
      back = 0;
#pragma unroll
      for (int i = 0; i < L::ACOP; ++i) {
        // piece c of row r at slot c ^ (r & 7); rows past the tile repeat its last
        const int cc = 64 * (L::ACOP * aw + i) + lane, r = cc / CPR, ch = (cc % CPR) ^ (r & 7);
        off[i] = (uint32_t)min(r, it.rows - 1) * (uint32_t)arow + 16 * ch;
        back |= (uint32_t)(ch >= CPR / 2) << i;
      }
#pragma unroll
      for (int i = 0; MXA && i < L::AGCOP; ++i) {
        const int r = SHORT ? 16 * (L::AGCOP * aw + i) + (lane >> 2) : 32 * aw + (lane >> 1);
        soff[i] = (uint32_t)min(r, it.rows - 1) * (uint32_t)srow;
      }
    }
    const int s = it.s0 + ls;
    const bool fresh = MXA && ls % kGroupStages == 0;
    if (fresh) {
      ++group;
      const uint32_t buf = lds0 + L::AS + (group % L::BUFS) * L::ASB;
#pragma unroll
      for (int i = 0; i < L::AGCOP; ++i) {
        if (SHORT) lds_copy4(sb + soff[i] + min(4 * (lane & 3), srow - 4), buf + 256 * (L::AGCOP * aw + i));
        else lds_copy16_s(sb, soff[i] + (uint32_t)scale_at(s, lane & 1, srow), buf + 1024 * aw);
      }
    }
    const uint32_t base = lds0 + (g % L::NST) * L::STAGE + L::S_B;
    const uint8_t* as = ab + (int64_t)s * L::AROW;
    if (half && s == sc.stages - 1) {
#pragma unroll
      for (int i = 0; i < L::ACOP; ++i)
        lds_copy16_s(as, off[i] - (back >> i & 1 ? L::AROW / 2 : 0), base + 1024 * (L::ACOP * aw + i));
    } else {
#pragma unroll
      for (int i = 0; i < L::ACOP; ++i) lds_copy16_s(as, off[i], base + 1024 * (L::ACOP * aw + i));
    }
    if (++ls == it.ns) {
      ls = 0;
      ++li;
    }
    return fresh;
  };
  copy_loop<L::NST, L::ACOP, L::AGCOP, L::template IN_FLIGHT<L::ACOP, L::AGCOP>>(sc, issue);
}

// One 128-K half h of a stage: acc[m][n] += W(column tile n) A(sub-tile m)^T for
// the first nm sub-tiles (FULL: all of them, with no branches between their reads)
template <bool MXA, int WF, int SUB, bool SHORT, bool FULL>
__device__ __forceinline__ void mul_half(v4f (&acc)[SUB][2], const uint8_t* bs, const uint8_t* as, const uint8_t* ws,
                                         const uint8_t* xs, int h, int w, int g, int r, int nm) {
  using L = Lay<MXA, WF, SUB, SHORT>;
  const int blk = 4 * h + g;
  uint32_t b[2][6], wsc[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int jr = 32 * w + 16 * n + r;
    wsc[n] = ws[L::GROW * jr + blk];
    if (WF == 1) {
      const uint4 v = *(const uint4*)(bs + jr * L::BROW + 16 * (blk ^ (jr & 7)));
      b[n][0] = v.x; b[n][1] = v.y; b[n][2] = v.z; b[n][3] = v.w; b[n][4] = 0; b[n][5] = 0;
    } else {
      // 24 bytes: a 16-byte piece and half of one, which follows it where g is even and
      // precedes it where g is odd.  (Both kinds of lane read at once; a branch for each
      // and no turn: 16-row tiles 607 against 557 us over 384 experts, 64-row tiles 102
      // against 81, MXFP8 94 against 66 over 1024 x 4096 x 7168.)
      const uint8_t* q = bs + jr * L::BROW;
      const bool odd = g & 1;
      int cv = (3 * blk + 1) / 2 + turn(jr), cd = (odd ? (3 * blk) / 2 : 3 * blk / 2 + 1) + turn(jr);
      cv -= cv >= 12 ? 12 : 0;
      cd -= cd >= 12 ? 12 : 0;
      const uint4 v = *(const uint4*)(q + 16 * cv);
      const uint2 d = *(const uint2*)(q + 16 * cd + (odd ? 8 : 0));
      b[n][0] = odd ? d.x : v.x;
      b[n][1] = odd ? d.y : v.y;
      b[n][2] = odd ? v.x : v.z;
      b[n][3] = odd ? v.y : v.w;
      b[n][4] = odd ? v.z : d.x;
      b[n][5] = odd ? v.w : d.y;
    }
  }
  // a lane's part of sub-tile m: its row's block
  auto row = [&](int m, int piece) {
    return *(const uint4*)(as + (16 * m + r) * L::AROW + 16 * (piece ^ (r & 7)));
  };
  if (MXA) {
#pragma unroll
    for (int m = 0; m < SUB; ++m) {
      if (!FULL && m >= nm) continue;
      const uint4 lo = row(m, 8 * h + g), hi = row(m, 8 * h + 4 + g);
      const v8i av = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      const int asc = (int)xs[L::GROW * (16 * m + r) + blk];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const v8i bv = {(int)b[n][0], (int)b[n][1], (int)b[n][2], (int)b[n][3], (int)b[n][4], (int)b[n][5], 0, 0};
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc[m][n], Fmt<WF>::MFMA, 0, 0,
                                                                     (int)wsc[n], 0, asc);
      }
    }
    return;
  }
  // eight k at a time, so that the conversions of the next run beside the MFMAs
  // of these
  const float sc[2] = {e8m0_to_f32(wsc[0]), e8m0_to_f32(wsc[1])};
  v32bf wide[2];
  if (WF == 2) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      wide[n] = __builtin_amdgcn_cvt_scalef32_pk32_bf16_bf6(
          (v6i){(int)b[n][0], (int)b[n][1], (int)b[n][2], (int)b[n][3], (int)b[n][4], (int)b[n][5]}, sc[n]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v8bf bv[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (WF == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) bv[n][i] = wide[n][8 * k + i];
      } else {
        const v2bf q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b[n][k], sc[n], 0);
        const v2bf q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b[n][k], sc[n], 1);
        const v2bf q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b[n][k], sc[n], 2);
        const v2bf q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b[n][k], sc[n], 3);
        bv[n] = (v8bf){q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
      }
    }
#pragma unroll
    for (int m = 0; m < SUB; ++m) {
      if (!FULL && m >= nm) continue;
      const uint4 a = row(m, 4 * blk + k);
      v8bf av;
      __builtin_memcpy(&av, &a, 16);
#pragma unroll
      for (int n = 0; n < 2; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], av, acc[m][n], 0, 0, 0);
    }
  }
}

template <bool MXA, int WF, int SUB, bool SHORT>
__device__ __forceinline__ void multiply(const FcArgs& p, const Sched& sc, const uint8_t* smem, int w) {
  using L = Lay<MXA, WF, SUB, SHORT>;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int srow = p.K / 32;
  const bool half = p.K % RK != 0;
  v4f acc[SUB][2];
#pragma unroll
  for (int m = 0; m < SUB; ++m) acc[m][0] = acc[m][1] = (v4f){0.f, 0.f, 0.f, 0.f};
  // The epilogue's operands are requested when the item starts; with 64 rows and
  // short K, whose items have one stage or two, an item ahead (8192 x 4096 x 256 E2M1
  // x bf16: 79 against 94 us; the other kernels lose 2 to 10% by it).
  constexpr bool kAhead = SUB > 1 && SHORT;
  Item it = {}, next = {};
  EpiIn in[SUB], next_in[SUB];
  EpiBias bias = {}, next_bias = {};
  int li = 0, ls = 0, group = -1, gs = 0, col = 0, nm = 1;  // gs: the group's first stage
  // the lane holds a piece of out per sub-tile: its row r, columns 8g .. 8g + 7
  // of the wave's 32
  auto column = [&](const Item& i) { return i.nb * RN + 32 * w + 8 * g; };
  auto mine = [&](const Item& i, int m, int c) { return 16 * m + r < i.rows && c < p.N; };
  auto at = [&](const Item& i, int m, int c) { return (int64_t)(i.p0 + 16 * m + r) * p.N + c; };
  auto request = [&](const Item& i, EpiIn (&to)[SUB], EpiBias& b) {
    if (sc.S > 1) return;  // (launch_linear_join's)
    const int c = column(i);
#pragma unroll
    for (int m = 0; m < SUB; ++m)
      if (mine(i, m, c)) to[m] = epi_in(p.epi, at(i, m, c));
    if (c < p.N) b = epi_bias(p.epi, p.N, i.expert, c);
  };
  if (kAhead) {
    next = item_at<L::RM>(p, sc, 0);
    request(next, next_in, next_bias);
  }
  for (int gi = 0; gi < sc.total; ++gi) {
    if (ls == 0) {
      if (kAhead) {
        it = next;
        bias = next_bias;
#pragma unroll
        for (int m = 0; m < SUB; ++m) in[m] = next_in[m];
        if (li + 1 < sc.items) {
          next = item_at<L::RM>(p, sc, li + 1);
          request(next, next_in, next_bias);
        }
      } else {
        it = item_at<L::RM>(p, sc, li);
        request(it, in, bias);
      }
      nm = (it.rows + 15) >> 4;
      col = column(it);
    }
    const int s = it.s0 + ls;
    if (ls % kGroupStages == 0) {
      ++group;
      gs = s;
    }
    wait_lgkm0();
    barrier();
    const uint8_t* st = smem + (gi % L::NST) * L::STAGE;
    // scale byte of block b of the stage: [GROW row + b]
    const int h = (s - gs) >> 1, so = SHORT ? 8 * s : 16 * h + 8 * s - scale_at(gs, h, srow);
    const uint8_t* ws = smem + L::WS + (group % L::BUFS) * L::WSB + so;
    const uint8_t* xs = smem + L::AS + (group % L::BUFS) * L::ASB + so;
    // A whole stage of a whole tile in one block lets the two halves' LDS reads and
    // conversions run together: 16-row E3M2 x bf16 8% faster, 64-row tiles up to 5%; the
    // others of 16 rows lose 3% by it and take a branch between.
    const bool two = !(half && s == sc.stages - 1);
    if (SUB == 1 && (MXA || WF == 1)) {
      mul_half<MXA, WF, SUB, SHORT, true>(acc, st, st + L::S_B, ws, xs, 0, w, g, r, nm);
      if (two) mul_half<MXA, WF, SUB, SHORT, true>(acc, st, st + L::S_B, ws, xs, 1, w, g, r, nm);
    } else if ((SUB == 1 || nm == SUB) && two) {
      mul_half<MXA, WF, SUB, SHORT, true>(acc, st, st + L::S_B, ws, xs, 0, w, g, r, nm);
      mul_half<MXA, WF, SUB, SHORT, true>(acc, st, st + L::S_B, ws, xs, 1, w, g, r, nm);
    } else {
      mul_half<MXA, WF, SUB, SHORT, false>(acc, st, st + L::S_B, ws, xs, 0, w, g, r, nm);
      if (two) mul_half<MXA, WF, SUB, SHORT, false>(acc, st, st + L::S_B, ws, xs, 1, w, g, r, nm);
    }
    if (++ls < it.ns) continue;
#pragma unroll
    for (int m = 0; m < SUB; ++m) {
      if (mine(it, m, col)) {
        if (sc.S > 1) {
          // a K range's sums, for launch_linear_join
          const int ks = (sc.q + li * sc.Q) % sc.S;
          float4* part = (float4*)(p.part + (int64_t)ks * p.dense_rows * p.N + at(it, m, col));
          part[0] = make_float4(acc[m][0][0], acc[m][0][1], acc[m][0][2], acc[m][0][3]);
          part[1] = make_float4(acc[m][1][0], acc[m][1][1], acc[m][1][2], acc[m][1][3]);
        } else {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[m][i >> 2][i & 3] + epi_bias_at(p.epi, bias, i);
          epi_store(p.epi, at(it, m, col), in[m], v);
        }
      }
      acc[m][0] = acc[m][1] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    ls = 0;
    ++li;
  }
}

template <bool MXA, int WF, int SUB, bool SHORT>
__global__ __launch_bounds__(rows_threads(SUB), 1) void k_linear_rows(FcArgs p) {
  using L = Lay<MXA, WF, SUB, SHORT>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[L::TOTAL];
  Sched sc;
  sc.S = p.ksplit > 1 ? p.ksplit : 1;
  sc.NB = p.nchunks;
  sc.stages = (p.K + RK - 1) / RK;
  const int ntiles = p.dense_rows > 0 ? (p.dense_rows + L::RM - 1) / L::RM : *p.num_tiles;
  sc.Q = gridDim.x;
  // Workgroups b, b + 8, .. share an XCD's L2 (11824 rows over 75 experts, 240 x 2944
  // E2M1 x MXFP8: 50 against 55 us).  Where the column blocks of a tile
  // go round the XCDs evenly and each XCD has two or more, items are dealt out in
  // turn, and an XCD keeps its columns' weights for all tiles; otherwise an XCD takes
  // neighbouring items, so that the tiles' rows are read by one XCD or two.
  sc.q = (sc.NB % 8 == 0 && sc.NB >= 16) || sc.Q % 8 ? blockIdx.x : (blockIdx.x & 7) * (sc.Q >> 3) + (blockIdx.x >> 3);
  const int nitems = ntiles * sc.NB * sc.S;
  sc.items = nitems > sc.q ? (nitems - sc.q + sc.Q - 1) / sc.Q : 0;
  sc.total = 0;
  if (sc.S == 1) {
    sc.total = sc.items * sc.stages;
  } else {
    for (int li = 0; li < sc.items; ++li) {
      const int ks = (sc.q + li * sc.Q) % sc.S;
      sc.total += range0(sc, ks + 1) - range0(sc, ks);
    }
  }
  if (sc.total == 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w < kMulWaves) multiply<MXA, WF, SUB, SHORT>(p, sc, smem, w);
  else if (w < kWaveA) copy_weights<MXA, WF, SUB, SHORT>(p, sc, smem, w - kMulWaves);
  else copy_rows<MXA, WF, SUB, SHORT>(p, sc, smem, w - kWaveA);
}

// The sums of a split call's K ranges, in ascending order, and its epilogue: a
// piece of 8 columns per thread.
__global__ __launch_bounds__(64) void k_linear_join(FcArgs p, int64_t n8) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n8) return;
  const EpiIn in = epi_in(p.epi, 8 * i);
  const EpiBias bias = epi_bias(p.epi, p.N, 0, (int)(8 * i % p.N));
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < p.ksplit; ++k) {
    const float4* v = (const float4*)p.part + 2 * (k * n8 + i);
    const float4 lo = v[0], hi = v[1];
    const float a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] += a[q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) s[q] += epi_bias_at(p.epi, bias, q);
  epi_store(p.epi, 8 * i, in, s);
}

}  // namespace

template <int SUB, bool SHORT>
static hipError_t launch_rows_t(const FcArgs& p, bool mx_act, int wfmt, int grid, hipStream_t st) {
  if (mx_act && wfmt == 1) k_linear_rows<true, 1, SUB, SHORT><<<grid, rows_threads(SUB), 0, st>>>(p);
  else if (mx_act) k_linear_rows<true, 2, SUB, SHORT><<<grid, rows_threads(SUB), 0, st>>>(p);
  else if (wfmt == 1) k_linear_rows<false, 1, SUB, SHORT><<<grid, rows_threads(SUB), 0, st>>>(p);
  else k_linear_rows<false, 2, SUB, SHORT><<<grid, rows_threads(SUB), 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_linear_rows(const FcArgs& p, bool mx_act, int wfmt, int rows, int grid, hipStream_t st) {
  if (grid < 1) grid = 1;
  // a K range has two stages at least, as the scale buffers assume
  if (p.K < 128 || p.K > kMaxK || p.K % 128 || (rows != 16 && rows != 64)) return hipErrorInvalidValue;
  if (p.ksplit > 1 && (p.K + RK - 1) / RK < 2 * p.ksplit) return hipErrorInvalidValue;
  if (p.K < 512)
    return rows == 16 ? launch_rows_t<1, true>(p, mx_act, wfmt, grid, st)
                      : launch_rows_t<4, true>(p, mx_act, wfmt, grid, st);
  return rows == 16 ? launch_rows_t<1, false>(p, mx_act, wfmt, grid, st)
                    : launch_rows_t<4, false>(p, mx_act, wfmt, grid, st);
}

hipError_t launch_linear_join(const FcArgs& p, hipStream_t st) {
  const int64_t n8 = (int64_t)p.dense_rows * p.N / 8;
  k_linear_join<<<(unsigned)((n8 + 63) / 64), 64, 0, st>>>(p, n8);
  return hipGetLastError();
}

}  // namespace moe_mx
