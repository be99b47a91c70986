// Choice of the kernel of an mx_linear call and the layout of its workspace: host
// code on sizes alone, which a test compiles and asks as well.
#pragma once
#include <algorithm>
#include <cmath>

#include "gemm.h"
#include "internal.h"

namespace moe_mx {

// GEMM kernel family of one FC1/FC2 pair or of one mx_linear call
enum class Fc { kStream, kSmall, kMid, kTiled, kWide, kFew, kRows };

inline int wbits(mx_elem_t f) { return f == MX_E2M1 ? 4 : (f == MX_E3M2 ? 6 : 8); }

inline size_t gemm_quant_bytes(int64_t M, int64_t K) {
  return align_up((size_t)(M * K), 256) + align_up((size_t)(M * K / 32), 256);
}

// Kernel, tile height and workspace layout of one mx_linear call.
struct LinearPlan {
  Fc kind;
  int rows;        // M-tile height
  int max_tiles;   // grouped: room of the tile list
  int ksplit;      // kRows, dense: K ranges (0 or 1: none)
  size_t quant, tiles, ntiles, part, total;
};

inline bool linear_sizes_ok(const mx_linear_problem_t& p) {
  return p.M >= 0 && p.N > 0 && p.K > 0 && p.K % 32 == 0 && p.groups >= 0 && p.groups <= kMaxExperts &&
         p.w_stride >= 0 && p.w_scale_stride >= 0;
}
inline bool linear_supported(const mx_linear_problem_t& p) {
  // the bounds keep tile counts and per-workgroup step counts inside 32 bits
  return p.w_fmt != MX_E4M3 && p.N % 8 == 0 && p.K % 128 == 0 && p.M <= (int64_t)1 << 30 && p.N <= (int64_t)1 << 30 &&
         p.K <= kMaxK && (double)p.M * p.N <= 34359738368.0 &&
         (double)p.M * p.N * p.K <= 4503599627370496.0;
}

// Choice of the kernel: the smallest of the estimated times below, in
// microseconds, which follow the kernels' structure: items over kLinearWgs
// workgroups, rounds of them, steps of K per item, a measured time per step and one
// per item for its epilogue (MI355X; without what every call pays for its launch):
//   few rows (gemm_few.hip; 16 x 16 items, 1024 K a step)  E2M1 x bf16: 1 row 0.43,
//     16 rows 1.0; E3M2 0.2 more; MXFP8 0.4 more, 0.8 up to K = 1024 (it quantizes in
//     place); twice that with groups, whose weights come from HBM (184 rows over 69
//     experts, 1840 x 896: 42 us, 16-row tiles 21)
//   rows (gemm_rows.hip; 256 K a step)  16 x 128 items: E2M1 0.55, E3M2 0.75
//     (bf16), 0.6;
//     64 x 128 items: E2M1 1.1 (bf16), 0.75 (MXFP8), E3M2 1.3, 0.95; 1.15
//     times that with groups
//   mid (E2M1 x bf16; 128 K a step)  64 x 256 items 1.06, 128 x 256 1.6
//   tiled (MXFP8)  128 x 256 items 1.08, E3M2 1.2; 192 x 128 0.88, 1.1
//   wide (E2M1 x MXFP8)  192 x 256 items 1.27
//   epilogues with a residual: 13.6 us per 128 x 256 item of mid, 9.6 of tiled, 18 of
//     wide's, 4.3 of 64 x 128 (8192 x 4096, K = 1024 and 7168)
// E.g. 64 rows of bf16 x E2M1, N = 4096, K = 7168: few 40, 16-row tiles in two K
// ranges 16.1, 64-row tiles in four 16.5, mid 66; 8192 rows: 64-row tiles 547, mid
// 433; 8192 rows of MXFP8 x E2M1: K = 7168 wide 276, tiled 288; K = 1024 wide 93, tiled
// 81.  A call that streams every expert's weights is bound by that (kWeightRate).
// Sizes only, so that the workspace does not depend on the device.
constexpr int kLinearWgs = 256;
constexpr double kWeightRate = 5.2e6;  // bytes per microsecond from HBM

struct LinearCost {
  const mx_linear_problem_t& p;
  double active;   // groups with rows (expected)
  double per;      // rows of one of them
  bool quant;      // bf16 rows to MXFP8 by a kernel of its own, where one is needed

  LinearCost(const mx_linear_problem_t& q, bool has_a_scale) : p(q), quant(q.act == MOE_ACT_MXFP8 && !has_a_scale) {
    if (p.groups > 0) {
      active = p.groups * (1.0 - std::pow(1.0 - 1.0 / p.groups, (double)p.M));
      active = std::max(active, 1.0);
    } else {
      active = 1.0;
    }
    per = p.M / active;
  }
  double tiles(int bm) const {
    if (p.groups == 0) return std::ceil(p.M / (double)bm);
    return active * std::max(1.0, per / bm + 0.5);
  }
  // items of bm rows and bn columns in `ksplit` K ranges, `steps` of `t` each
  double time(int bm, int bn, double steps, double t, int ksplit = 1) const {
    const double items = tiles(bm) * std::ceil(p.N / (double)bn) * ksplit;
    double rounds = items / kLinearWgs;
    if (p.groups == 0 || rounds < 8.0) rounds = std::ceil(rounds);  // (else the tile count is too rough)
    const double weights = active * p.N * (double)p.K * (wbits(p.w_fmt) / 8.0 + 1.0 / 32.0) / kWeightRate;
    return std::max(rounds * (std::ceil(steps / ksplit) * t + 1.0 + 0.3 / 1024.0 * bm * bn), weights);
  }
  // launches in front of a kernel: the tile list and the quantized activations
  double before() const {
    return (p.groups > 0 ? 4.0 : 0.0) + (quant ? 3.5 + (double)p.M * p.K * 3.0 / 3.5e6 : 0.0);
  }
  double join_time(int ksplit) const { return ksplit > 1 ? 4.5 + (double)ksplit * p.M * p.N * 8.0 / 4.0e6 : 0.0; }
};

// M-tiles of bm rows that a call can have, whatever its offsets
inline int64_t most_tiles(const mx_linear_problem_t& p, int bm) {
  if (p.groups == 0) return (p.M + bm - 1) / bm;
  return p.M / bm + std::min(p.M, (int64_t)p.groups);
}

inline void linear_kind(const mx_linear_problem_t& p, bool has_a_scale, LinearPlan& f) {
  const LinearCost c(p, has_a_scale);
  const bool e2m1 = p.w_fmt == MX_E2M1, mx = p.act == MOE_ACT_MXFP8;
  double best = -1.0;
  auto take = [&](Fc kind, int rows, int ksplit, double us) {
    if (best >= 0.0 && us >= best) return;
    best = us;
    f.kind = kind;
    f.rows = rows;
    f.ksplit = ksplit;
  };
  // (its grid has one workgroup per item: as many as its launch can have, of the most
  // tiles there can be)
  const int64_t blocks = (p.N + kFewCols - 1) / kFewCols;
  if (most_tiles(p, kStreamRows) * blocks <= 1 << 20) {
    const double more = (e2m1 ? 0.0 : 0.2) + (!mx ? 0.0 : p.K <= 1024 ? 0.8 : 0.4);
    const double t = (p.groups > 0 ? 2.0 : 1.0) * (0.43 + 0.57 * std::min(c.per, 16.0) / 16.0 + more);
    // (with bf16 several of its workgroups share a CU: no whole rounds; each finds
    // its tile in the offsets)
    const double steps = p.K <= 1024 ? 1.0 : std::ceil(p.K / 2048.0) * 2.0;
    const double rounds = std::max(1.0, c.tiles(16) * blocks / kLinearWgs);
    const double find = p.groups > 0 ? 1.5 : 0.0;
    take(Fc::kFew, kStreamRows, 0, mx ? c.time(16, 16, steps, t) : 1.0 + rounds * (t * steps + find));
  }
  const double stages = std::ceil(p.K / (double)kRowsK);
  const double own = p.groups > 0 ? 1.15 : 1.0;  // groups share no weights in the caches
  const double t16 = own * (e2m1 ? 0.55 : mx ? 0.6 : 0.75), t64 = own * (e2m1 ? (mx ? 0.75 : 1.1) : (mx ? 0.95 : 1.3));
  // K ranges of at least two stages, dense calls only
  const int most = p.groups > 0 ? 1 : (int)std::min(16.0, std::max(1.0, std::floor(stages / 2.0)));
  for (int s = 1; s <= most; ++s) {
    const double more = c.before() + c.join_time(s);
    take(Fc::kRows, 16, s, c.time(16, kRowsCols, stages, t16, s) + more);
    take(Fc::kRows, 64, s, c.time(64, kRowsCols, stages, t64, s) + more);
  }
  // (whole scale groups of 512 K)
  if (p.K < kMidK) return;
  const double steps = std::ceil(p.K / (double)kMidK) * (kMidK / 128);
  if (!mx && e2m1) {
    take(Fc::kMid, kMidRows, 0, c.time(kMidRows, kWideCols, steps, 1.06) + c.before());
    take(Fc::kMid, kMidRowsHigh, 0, c.time(kMidRowsHigh, kWideCols, steps, 1.6) + c.before());
  }
  if (mx) {
    take(Fc::kTiled, kTiledRowsLow, 0,
         c.time(128, tiled_weight_rows(kTiledRowsLow), steps, e2m1 ? 1.08 : 1.2) + c.before());
    take(Fc::kTiled, kTiledRows, 0,
         c.time(192, tiled_weight_rows(kTiledRows), steps, e2m1 ? 0.88 : 1.1) + c.before());
    // (its 32-bit offsets into A, and column blocks of 64 inside N)
    if (e2m1 && p.K >= 1024 && p.K % kTiledKMultiple == 0 && p.N % 64 == 0 && (double)p.M * p.K < 4294967296.0)
      take(Fc::kWide, kTiledRows, 0, c.time(192, kWideCols, steps, 1.27) + c.before());
  }
}

inline LinearPlan linear_plan(const mx_linear_problem_t& p, bool has_a_scale) {
  LinearPlan f = {};
  linear_kind(p, has_a_scale, f);
  if (p.groups > 0) f.max_tiles = (int)most_tiles(p, f.rows);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = align_up(o + bytes, 256);
    return r;
  };
  if (p.act == MOE_ACT_MXFP8 && !has_a_scale && f.kind != Fc::kFew) f.quant = take(gemm_quant_bytes(p.M, p.K));
  if (p.groups > 0 && f.kind != Fc::kFew) {
    f.tiles = take((size_t)f.max_tiles * sizeof(Tile));
    f.ntiles = take(4);
  }
  if (f.ksplit > 1) f.part = take((size_t)f.ksplit * p.M * p.N * 4);
  f.total = o;
  return f;
}

}  // namespace moe_mx
