// Arguments of the grouped FC1 / FC2 kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace moe_mx {

// Bias of mx_linear: none, fp32 or bf16 rows on 16-byte addresses, or on any
constexpr int kBiasNone = 0, kBiasF32 = 1, kBiasBf16 = 2, kBiasF32Any = 3, kBiasBf16Any = 4;

// Epilogue operands of mx_linear (epilogue.h); null: absent
struct Epilogue {
  const void* bias;          // [groups, N] as bias_kind says
  int bias_kind;             // kBias*
  int fn;                    // mx_fn_t
  const uint16_t* mul;       // [M, N] bf16
  const uint16_t* residual;  // [M, N] bf16
  __bf16* out;               // [M, N]
};

struct FcArgs {
  // M-tiles: routed mode reads `tiles[0 .. *num_tiles)`, grid sized for max_tiles;
  // dense mode (dense_rows > 0) covers rows [0, dense_rows) of a single expert.
  const Tile* tiles;
  const int32_t* num_tiles;
  int max_tiles;
  int dense_rows;
  // mx_linear's few-row kernel: no tile list, but the offsets of `groups` groups
  // over group_rows rows
  const int32_t* group_offsets;
  int groups, group_rows;
  // routed rows: permuted position p -> assignment a = t*k + j
  const int32_t* sorted_assign;
  int k;
  uint32_t kdiv;       // k > 1: ceil(2^32 / k), so that the token of assignment a is
                       // umulhi(a, kdiv), exact while a*k < 2^32
  const float* topk_w;  // FC2 routed: weight of assignment a
  const float* sorted_w;  // routed: weight of permuted row p (= topk_w[sorted_assign[p]])
  float dense_weight;   // FC2 dense: weight of every row
  // A operand: FC1 -> x rows (bf16 [T, K] or E4M3 codes [T, K] + scales [T, K/32]),
  //            FC2 -> h rows in permuted order (bf16 [P, K] or codes + scales)
  const void* a;
  const uint8_t* a_scale;
  // B operand: weights [experts, N_w, K*bits/8] + scales [experts, N_w, K/32]
  const uint8_t* w;
  const uint8_t* w_scale;
  int64_t w_estride;   // bytes per expert
  int64_t ws_estride;  // scale bytes per expert
  int act_fn;          // FC1: gated activation (moe_act_fn_t; 0 = SiLU)
  int K;               // contraction length (H for FC1, I for FC2)
  int N;               // FC1: I (h columns); FC2: H
  int nchunks;         // column chunks of N per M-tile
  // outputs
  void* out;           // FC1: h (bf16 [P, I] or E4M3 codes [P, I])
  uint8_t* out_scale;  // FC1 MX: h scales [P, I/32]
  uint16_t* obuf;      // FC2: bf16 rows [A, N] (routed: row = assignment a, holding
                       // w(a) * o; dense: row = token, holding dense_weight * o),
                       // the product taken in fp32 and rounded once (RNE)
  // dense FC2 on the small-M kernel only: K split into ksplit equal ranges
  // (ksplit > 1), each item writing its unscaled fp32 sum to part
  // [ksplit, dense_rows, N] instead of obuf; 0 or 1 = no split
  int ksplit;
  float* part;
  // few-token FC1 on the small-M kernel (launch_fc_small_routed): every
  // workgroup routes the batch itself from the router logits [T, E] (local
  // experts [off, off + L)) instead of reading tiles, num_tiles and
  // sorted_assign, and workgroup 0 writes the routing out as the routing and
  // permutation kernels would: ids_out / w_out [T, k], offsets_out [L + 1],
  // sorted_out / sorted_w_out (the permuted assignments and their weights),
  // tiles_out and ntiles_out (one tile per active local expert)
  const float* logits;
  int T, E, off, L;
  int32_t* ids_out;
  float* w_out;
  int32_t* offsets_out;
  int32_t* sorted_out;
  float* sorted_w_out;
  Tile* tiles_out;
  int32_t* ntiles_out;
  // mx_linear on the FC2 kernels: rows of A and of the output are permuted rows
  // (no sorted_assign, no row weights), finished by the epilogue
  bool linear;
  Epilogue epi;
};

// The checks that mx_linear and mx4_linear share (everything but the workspace and the device;
// M == 0 passes without its tensors), and the kernel arguments they begin with: epilogue,
// weights, activations as given.
struct LinearCall {
  int64_t w_stride, s_stride;  // bytes between the groups' matrices and scales
};
moe_status_t check_linear(const mx_linear_problem_t& p, const mx_linear_tensors_t& t, LinearCall& call);
FcArgs linear_args(const mx_linear_problem_t& p, const mx_linear_tensors_t& t, const LinearCall& call);
// compute units of the current device, for persistent grids
int device_cus();

// Columns of N covered by one wave of the stream kernels.
constexpr int kStreamColsFc1 = 32;
constexpr int kStreamColsFc2 = 64;
constexpr int kStreamRows = 16;

hipError_t launch_fc_stream(const FcArgs& p, bool fc1, bool mx_act, int wfmt, hipStream_t st);

// Tiled variant (MXFP8 activations): M-tiles of up to `rows` rows (kTiledRows,
// or kTiledRowsLow when experts see fewer rows: less LDS for activations,
// room for wider N-blocks), N-blocks of tiled_weight_rows(rows) weight rows,
// i.e. half as many h columns (FC1: nchunks = I / (that / 2)) or that many
// output columns (FC2: nchunks = H / that); `grid` persistent workgroups
// (rounded down to a multiple of 8, at least 8).  Requires K to be a multiple
// of kTiledKMultiple (scales travel in groups of 4 128-K stages; mx_linear: of 128,
// at least kTiledKMultiple).
constexpr int kTiledRows = 192;
constexpr int kTiledRowsLow = 128;
constexpr int kTiledKMultiple = 512;
// weight rows per N-block of the tiled kernel for M-tiles of `rows` rows
constexpr int tiled_weight_rows(int rows) { return rows == kTiledRowsLow ? 256 : 128; }
// N-blocks of the small-M kernel: 64 h columns (FC1) or 128 output columns (FC2)
constexpr int kSmallColsFc1 = 64;
constexpr int kSmallColsFc2 = 128;
hipError_t launch_fc_tiled(const FcArgs& p, bool fc1, int wfmt, int rows, int grid, hipStream_t st);

// Wide variant (MXFP8 activations x E2M1 weights): M-tiles of up to kTiledRows
// rows, N-blocks of kWideCols weight rows, i.e. 128 h columns (FC1: nchunks =
// I / 128) or 256 output columns (FC2: nchunks = H / 256); `grid` persistent
// workgroups (rounded down to a multiple of 8, at least 8).  Requires
// K % 128 == 0 and K >= 256.
constexpr int kWideCols = 256;
hipError_t launch_fc_wide(const FcArgs& p, bool fc1, int grid, hipStream_t st);

// Small-M variant for bf16 activations and E2M1 weights: M-tiles of up to
// kStreamRows rows (the same tile list as the stream kernels), N-blocks of 64
// h columns (FC1) or 128 output columns (FC2); `grid` persistent workgroups.
// Requires K % kSmallK == 0.
constexpr int kSmallK = 256;
hipError_t launch_fc_small(const FcArgs& p, bool fc1, int grid, hipStream_t st);
// FC1 of the small-M kernel with the routing of a batch of at most
// kSmallRoutedTokens tokens and kSmallRoutedAssign assignments in its prologue
// (p.logits and the routing outputs set; E <= kMaxExperts); the tile height is
// kStreamRows, one tile per active local expert.
constexpr int kSmallRoutedTokens = 16;
constexpr int kSmallRoutedAssign = 128;
hipError_t launch_fc_small_routed(const FcArgs& p, int grid, hipStream_t st);
// y = bf16_RNE(alpha * sum over s of part[s]) for the ksplit partial sums of a
// split dense GEMM, summed in ascending s; n4 = rows * N / 4 (N % 4 == 0)
hipError_t launch_splitk_reduce(const float* part, int ksplit, int64_t n4, float alpha, uint16_t* y,
                                hipStream_t st);

// mx_linear with few rows (gemm_few.hip): items of 16 rows and kFewCols columns
// (nchunks column blocks), one workgroup each; quant: bf16 activations are
// quantized to MXFP8 on the way.
constexpr int kFewCols = 16;
hipError_t launch_linear_few(const FcArgs& p, bool mx_act, bool quant, int wfmt, hipStream_t st);
// mx4_linear with a handful of rows, the same way: E2M1 codes, or (quant) bf16 rows quantized
// to them on the way.
hipError_t launch_mx4_few(const FcArgs& p, bool quant, hipStream_t st);
// mx_linear with weights through LDS (gemm_rows.hip): `grid` persistent
// workgroups, items of `rows` (16 or 64) rows and kRowsCols columns (nchunks column blocks),
// any K % 128 == 0.  Dense calls may split K's stages in
// p.ksplit ranges (p.part), joined by launch_linear_join.
constexpr int kRowsCols = 128;
constexpr int kRowsK = 256;
// mx_linear's largest K: 32-bit byte offsets over the rows of a tile of weights
constexpr int64_t kMaxK = (int64_t)1 << 24;
hipError_t launch_linear_rows(const FcArgs& p, bool mx_act, int wfmt, int rows, int grid, hipStream_t st);
hipError_t launch_linear_join(const FcArgs& p, hipStream_t st);

// Mid-M variant for bf16 activations and E2M1 weights when experts see many
// rows: M-tiles of up to `rows` rows (kMidRows or kMidRowsHigh), N-blocks of
// kWideCols weight rows, i.e. 128 h columns (FC1: nchunks = I / 128) or 256
// output columns (FC2: nchunks = H / 256); `grid` persistent workgroups
// (rounded down to a multiple of 8, at least 8).  Requires K % kMidK == 0
// (mx_linear: K % 128 == 0, K >= kMidK) and, for the FC1 gather, A*k < 2^32.
constexpr int kMidRows = 64;
constexpr int kMidRowsHigh = 128;
constexpr int kMidK = 512;
hipError_t launch_fc_mid(const FcArgs& p, bool fc1, int rows, int grid, hipStream_t st);

// mx4_linear with many rows (gemm_fp4.hip): `grid` persistent workgroups (rounded
// down to a multiple of 8, at least 8), items of `rows` (64, 128 or 256) rows and
// kFp4Cols columns.  Requires K % 128 == 0, K >= kFp4K (16 bytes of scales per row) and N <=
// kFp4MaxN (32-bit offsets into the 256 rows of a tile of out).
constexpr int kFp4Cols = 256;
constexpr int kFp4K = 512;
constexpr int64_t kFp4MaxN = (int64_t)1 << 22;
// Tiles of 64 rows, dense: with p.ksplit > 1 an item takes one of as many ranges of K and
// leaves fp32 sums in p.part, joined by launch_linear_join.  A range has fp4_range stages of
// 256 K, an even number (scales come by two stages) of 4 or more (the copies are 3 ahead); the
// last one what is left, 4 or more too.
__host__ __device__ inline int fp4_range(int stages, int ranges) { return ((stages + ranges - 1) / ranges + 1) & ~1; }
inline bool fp4_range_ok(int stages, int ranges) {
  const int len = fp4_range(stages, ranges);
  return len >= 4 && stages - len * (ranges - 1) >= 4;
}
hipError_t launch_linear_fp4(const FcArgs& p, int rows, int grid, hipStream_t st);

}  // namespace moe_mx
