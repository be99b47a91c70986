// Choice of the kernel of an mx4_linear call and the layout of its workspace: host code
// on sizes alone, which a test compiles and asks as well.
#pragma once
#include "linear_plan.h"

namespace moe_mx {

// kFew: gemm_few.hip, E2M1 codes or bf16 quantized on the way; kTile: gemm_fp4.hip;
// kWiden: E4M3 codes of the E2M1 ones (every E2M1 value is an E4M3 value, with the same
// scale) and mx_linear's kernels
enum class Fc4 { kFew, kTile, kWiden };

struct Mx4Plan {
  Fc4 kind;
  int rows;               // kTile: M-tile height
  int max_tiles;          // kFew, kTile, grouped: M-tiles there can be
  size_t codes, scales;   // E2M1 codes and scales of bf16 rows
  size_t wide;            // kWiden: E4M3 codes
  size_t tiles, ntiles;   // kTile, grouped: the tile list
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
// (linear_plan.h; N = 4096, K = 7168 on an MI355X, from codes unless said, with the
// launches in front):
//   few rows: 1 row 7.9, 16 rows 9.5, 32 rows 15.5; from bf16 9.7, 14.1, 25.7
//   tiles of 64, 128 and 256 rows: up to 64 rows 18.5, 25, 38; 256 rows 23, 31, 40; 1024 rows
//     26, 35, 45; 4096 rows 88, 73, 62; 8192 rows 166, 142, 120: a stage of 256 K takes 0.6, 0.85
//     and 1.3 where few workgroups have an item and 0.75, 1.25 and 2.1 where all do
//   widened: 16 rows 12.9, 32 rows 12.7, 64 rows 17, 256 rows 26, 1024 rows 54, 8192 rows 260
// Experts: 512 rows over 384, 7168 x 2048: widened 359, 64-row tiles 370, 128 449; 16384 rows
// over 256, 1536 x 5120: 324, 268, 261, 256-row tiles 292; 65536 over 128, 1536 x 4096: 529,
// 405, 352, 309.
inline Mx4Plan mx4_plan(const mx4_linear_problem_t& p, bool has_a_scale) {
  const mx_linear_problem_t q = as_mxfp8(p);
  const LinearCost c(q, true);
  Mx4Plan f = {};
  double best = -1.0;
  auto take = [&](Fc4 kind, int rows, double us) {
    if (best >= 0.0 && us >= best) return;
    best = us;
    f.kind = kind;
    f.rows = rows;
  };
  const double before = p.groups > 0 ? 4.0 : 0.0;
  const double quant = has_a_scale ? 0.0 : 3.0 + (double)p.M * p.K * 2.53 / 4.5e6;
  const double stages = std::ceil(p.K / 256.0), own = p.groups > 0 ? 1.15 : 1.0;
  const double widen = 3.0 + (double)p.M * p.K * 1.5 / 4.5e6 + before + quant;
  take(Fc4::kWiden, 0, widen + std::min(c.time(16, kRowsCols, stages, own * 0.6), c.time(64, kRowsCols, stages, own * 0.75)));
  if (p.K >= kFp4K && p.N <= kFp4MaxN) {
    const double few[3] = {0.6, 0.85, 1.3}, all[3] = {0.75, 1.25, 2.1};
    for (int i = 0; i < 3; ++i) {
      const int rows = 64 << i;
      const double items = c.tiles(rows) * std::ceil(p.N / (double)kFp4Cols);
      const double t = few[i] + (all[i] - few[i]) * std::min(1.0, items / kLinearWgs);
      take(Fc4::kTile, rows, c.time(rows, kFp4Cols, stages, t) + before + quant);
    }
  }
  const int64_t blocks = (p.N + kFewCols - 1) / kFewCols;
  if (most_tiles(q, kStreamRows) * blocks <= 1 << 20) {
    const double rows = std::min(c.per, 16.0) / 16.0;
    const double t = (p.groups > 0 ? 2.0 : 1.0) * (has_a_scale ? 0.45 + 0.2 * rows : 0.68 + 0.55 * rows);
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
  if (f.kind == Fc4::kWiden) {
    f.wide = room((size_t)(p.M * p.K));
    f.rest_bytes = linear_plan(q, true).total;
    f.rest = room(f.rest_bytes);
  }
  f.total = o;
  return f;
}

}  // namespace moe_mx
