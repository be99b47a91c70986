// Choice of the kernel of an mx4_linear call and the layout of its workspace: host code
// on sizes alone, which a test compiles and asks as well.
#pragma once
#include "linear_plan.h"

namespace moe_mx {

// kFew: gemm_few.hip, E2M1 codes or bf16 quantized on the way; kTile: gemm_fp4.hip, for few
// dense items in ranges of K;
// kWiden: E4M3 codes of the E2M1 ones (every E2M1 value is an E4M3 value, with the same
// scale) and mx_linear's kernels
enum class Fc4 { kFew, kTile, kWiden };

struct Mx4Plan {
  Fc4 kind;
  int rows;               // kTile: M-tile height
  int ksplit;             // kTile: ranges of K (0: one)
  int max_tiles;          // kFew, kTile, grouped: M-tiles there can be
  size_t codes, scales;   // E2M1 codes and scales of bf16 rows
  size_t wide;            // kWiden: E4M3 codes
  size_t tiles, ntiles;   // kTile, grouped: the tile list
  size_t part;            // kTile, ranges of K: their sums
  size_t rest, rest_bytes;  // kWiden: mx_linear's own workspace
  size_t total;
};

// the product as one of mx_linear: MXFP8 activations given as codes
inline mx_linear_problem_t as_mxfp8(const mx4_linear_problem_t& p) {
  mx_linear_problem_t q = {};
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.groups = p.groups;
  q.act = MOE_ACT_MXFP8;
  q.w_fmt = MX_E2M1;
  q.fn = p.fn;
  q.bias_dtype = p.bias_dtype;
  q.w_stride = p.w_stride;
  q.w_scale_stride = p.w_scale_stride;
  return q;
}

// The smallest of the estimated times in microseconds, as linear_kind chooses
// (linear_plan.h).  Over 82 measured shapes (1 to 76800 rows, dense and 8 to 384 groups) the
// choice costs 0.7 % more than the best kernel each time, 19 % at most, but for the four of them
// that take ranges of K, which were not among the kernels measured then.
//   few rows in place (a step of 1024 K): from codes 0.45 to 0.65, from bf16 to 0.75 up to 8 rows
//     and to 1.23 from there on; twice that with groups (N = 4096, K = 7168: 1 row 7.2, 16 rows
//     9.5, 32 rows 15.7; from bf16 7.2, 14.4, 25.7)
//   tiles of 64, 128 and 256 rows: a stage of 256 K 0.6, 0.85 and 1.3 where few workgroups
//     have an item and 0.76, 1.12 and 2.05 where all do, 15 and 8 % more for the smaller ones
//     with groups, which share no weights; 1.4, 3.3 and 9 an item beside its stages.  N = 4096,
//     K = 7168: 64 rows 20, 25, 39; 1024 rows 27, 32, 47; 8192 rows 183, 143, 121; 65536 rows
//     of 128 groups, 1536 x 4096: 420, 307, 287; 512 rows of 384 groups, 7168 x 2048: 378, 425, 587
//   widened: 64 rows 17, 256 rows 26, 1024 rows 54, 8192 rows 260; the two grouped 469 and 368
struct Fp4Cost {
  double few, all, group, item;
};
constexpr Fp4Cost kFp4Cost[3] = {{0.6, 0.76, 1.15, 1.4}, {0.85, 1.12, 1.08, 3.3}, {1.3, 2.05, 1.0, 9.0}};
constexpr double kFp4WeightRate = 5.5e6;  // bytes per microsecond from HBM

inline Mx4Plan mx4_plan(const mx4_linear_problem_t& p, bool has_a_scale) {
  const mx_linear_problem_t q = as_mxfp8(p);
  const LinearCost c(q, true);
  Mx4Plan f = {};
  double best = -1.0;
  auto take = [&](Fc4 kind, int rows, double us, int ksplit = 0) {
    if (best >= 0.0 && us >= best) return;
    best = us;
    f.kind = kind;
    f.rows = rows;
    f.ksplit = ksplit;
  };
  const double before = p.groups > 0 ? 4.0 : 0.0;
  const double quant = has_a_scale ? 0.0 : 3.0 + (double)p.M * p.K * 2.53 / 4.5e6;
  const double stages = std::ceil(p.K / 256.0), own = p.groups > 0 ? 1.15 : 1.0;
  double rows8 = -1.0;  // of the kernels for few rows of E4M3, in K ranges as linear_kind has them
  const int most = p.groups > 0 ? 1 : (int)std::min(16.0, std::max(1.0, std::floor(stages / 2.0)));
  for (int s = 1; s <= most; ++s) {
    const double t = std::min(c.time(16, kRowsCols, stages, own * 0.55, s), c.time(64, kRowsCols, stages, own * 0.75, s)) +
                     c.join_time(s);
    if (rows8 < 0.0 || t < rows8) rows8 = t;
  }
  take(Fc4::kWiden, 0, 3.0 + (double)p.M * p.K * 1.5 / 4.5e6 + before + quant + rows8);
  if (p.K >= kFp4K && p.N <= kFp4MaxN) {
    const double weights = c.active * p.N * (double)p.K * (0.5 + 1.0 / 32.0) / kFp4WeightRate;
    for (int i = 0; i < 3; ++i) {
      const Fp4Cost& f4 = kFp4Cost[i];
      const double items = c.tiles(64 << i) * std::ceil(p.N / (double)kFp4Cols);
      double rounds = items / kLinearWgs;
      const double t = f4.few + (f4.all - f4.few) * std::min(1.0, rounds);
      if (p.groups == 0 || rounds < 8.0) rounds = std::ceil(rounds);
      const double tiles = rounds * (stages * t * (p.groups > 0 ? f4.group : 1.0) + f4.item);
      take(Fc4::kTile, 64 << i, 1.5 + std::max(tiles, weights) + before + quant);
    }
    // ranges of K while all items have a workgroup of their own (K = 7168; 64-row tiles in one
    // range, in several, widened: 33 x 4096 20 us, 13.1, 16.3; 100 x 4096 21, 15.8, 18.2; 64 x 1032
    // 19, 11.8, 12.6; 500 x 520 19.5, 15.8, 18; 256 x 4096 23.5, 24.0)
    const double items = c.tiles(64) * std::ceil(p.N / (double)kFp4Cols);
    for (int s = 2; p.groups == 0 && s * items <= kLinearWgs && s <= 16; ++s)
      if (fp4_range_ok((int)stages, s)) {
        const double t = kFp4Cost[0].few + (kFp4Cost[0].all - kFp4Cost[0].few) * s * items / kLinearWgs;
        take(Fc4::kTile, 64, 1.5 + fp4_range((int)stages, s) * t + kFp4Cost[0].item + c.join_time(s) + before + quant, s);
      }
  }
  const int64_t blocks = (p.N + kFewCols - 1) / kFewCols;
  if (most_tiles(q, kStreamRows) * blocks <= 1 << 20) {
    const double rows = std::min(c.per, 16.0) / 16.0;
    const double a = has_a_scale ? 0.2 * rows : p.M <= 8 ? 0.6 * rows : 0.23 + 0.55 * rows;
    const double t = (p.groups > 0 ? 2.0 : 1.0) * (0.45 + a);
    const double steps = p.K <= 1024 ? 1.0 : std::ceil(p.K / 2048.0) * 2.0;
    take(Fc4::kFew, kStreamRows, c.time(16, 16, steps, t));
  }

  if (p.groups > 0 && f.kind != Fc4::kWiden) f.max_tiles = (int)most_tiles(q, f.rows);
  size_t o = 0;
  auto room = [&](size_t bytes) {
    const size_t r = o;
    o = align_up(o + bytes, 256);
    return r;
  };
  if (!has_a_scale && f.kind != Fc4::kFew) {
    f.codes = room((size_t)(p.M * p.K / 2));
    f.scales = room((size_t)(p.M * p.K / 32));
  }
  if (p.groups > 0 && f.kind == Fc4::kTile) {
    f.tiles = room((size_t)f.max_tiles * sizeof(Tile));
    f.ntiles = room(4);
  }
  if (f.ksplit > 1) f.part = room((size_t)f.ksplit * p.M * p.N * 4);
  if (f.kind == Fc4::kWiden) {
    f.wide = room((size_t)(p.M * p.K));
    f.rest_bytes = linear_plan(q, true).total;
    f.rest = room(f.rest_bytes);
  }
  f.total = o;
  return f;
}

}  // namespace moe_mx
