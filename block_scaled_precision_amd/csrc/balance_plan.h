// Launch shapes of moe_balance and its gradient and the layout of the workspace: host code
// on sizes alone, which a test compiles and asks as well.
#pragma once
#include <algorithm>
#include <type_traits>

#include "internal.h"

namespace moe_mx {

constexpr int kThreadsB = 256;
constexpr int kFinishThreads = 1024;  // of a workgroup of the second launch
// Tokens up to which the loss takes one launch of one workgroup, for up to
// kOneSeqs sequences
constexpr int kOneTokens = 128, kOneSeqs = 4;

// Chunks of a loss of up to kChunkRows rows each; longer ones have more chunks, so that no sum
// in fp32 has more than 64 rows (of 4 groups, at 64 lanes a row) and as many groups.
constexpr int kMaxChunks = 512, kChunkRows = 256;

// Lanes per row and pieces per lane: calls F with them as compile-time constants.  The loss
// spends its time on what a row costs beside its values, reductions and a logarithm, so that
// 16 lanes a row, four rows a wave, take it as far as their registers reach (65536 x 128: 16
// lanes 12.4 us, 32 lanes 15.5); the gradient moves more bytes and wants more loads under way.
template <bool LOSS, class F>
void for_row_shape(bool vec, int E, F f) {
#define MOE_ROW_SHAPE(V, L, P) \
  if (E <= V * L * P) return f(std::integral_constant<int, V>(), std::integral_constant<int, L>(), \
                               std::integral_constant<int, P>())
  if (vec && LOSS) {
    MOE_ROW_SHAPE(4, 16, 1);
    MOE_ROW_SHAPE(4, 16, 2);
    MOE_ROW_SHAPE(4, 16, 3);
    MOE_ROW_SHAPE(4, 16, 4);
    MOE_ROW_SHAPE(4, 16, 6);
    MOE_ROW_SHAPE(4, 32, 4);
    MOE_ROW_SHAPE(4, 32, 6);
    MOE_ROW_SHAPE(4, 32, 8);
  } else if (vec) {
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
  int cols, blocks;  // experts of a workgroup of the second launch, workgroups per sequence
  size_t sum_p, sum_c, sum_z, sum_n, part, part_z, arrived, total;
};

inline BalancePlan balance_plan(int32_t T, int32_t E, int32_t S) {
  BalancePlan f = {};
  f.one = T <= kOneTokens && S <= kOneSeqs;
  if (f.one) return f;
  f.rows = (int)std::min<size_t>(align_up(std::max<size_t>(((size_t)T + kMaxChunks - 1) / kMaxChunks, 1), 16), kChunkRows);
  f.chunks = (T + f.rows - 1) / f.rows;
  f.cols = f.chunks / S <= 64 ? 64 : 16;
  f.blocks = (E + f.cols - 1) / f.cols;
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
  f.part = take((size_t)S * f.blocks * 8);
  f.part_z = take((size_t)S * 8);
  f.arrived = take(4);
  f.total = o;
  return f;
}

inline bool balance_sizes_valid(int32_t T, int32_t E, int32_t k, int32_t S) {
  return T >= 0 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= E && S >= 1;
}
// (A launch has fewer than 2^32 threads.  The second one's workgroups have 1024: S + S E / 64 of
// them with 64 experts each, S + S E / 16 with 16, which takes more than 64 chunks a sequence, so
// S < 2^16.)
inline bool balance_sizes_supported(int32_t T, int32_t E, int32_t k, int32_t S) {
  return (int64_t)T * k <= (int64_t)1 << 30 && T <= 1 << 30 && S <= 1 << 20 && (int64_t)S * E <= (int64_t)1 << 27;
}

// Rows of a group of lanes in the gradient, of which a workgroup has G: one where that leaves
// the chip room, more once there are workgroups enough (16, or as many as keep a launch at 2^23
// of them: it has fewer than 2^32 threads); and those workgroups
inline int balance_grad_rows(int64_t T, int64_t G) {
  const int64_t room = std::min<int64_t>(16, std::max<int64_t>(1, T / (G * 2048))), most = G << 23;
  return (int)std::max(room, (T + most - 1) / most);
}
inline int64_t balance_grad_blocks(int64_t T, int64_t G) {
  const int64_t rows = G * balance_grad_rows(T, G);
  return (T + rows - 1) / rows;
}

}  // namespace moe_mx
