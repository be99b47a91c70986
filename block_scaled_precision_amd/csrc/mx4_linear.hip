// mx4_linear: the matrix product with MXFP4 operands on both sides and mx_linear's
// epilogue (mxfp6-sm120 page, table of paths, "Dense" row, and "Execution model";
// TokenSpeed SiTU page, "Supported contract": MxE2m1).  Host side: validation, the choice of
// the kernel (mx4_plan.h) and the launches.
#include <hip/hip_runtime.h>

#include "gemm.h"
#include "internal.h"
#include "mx4_plan.h"

using namespace moe_mx;

extern "C" size_t mx4_linear_workspace_bytes(const mx4_linear_problem_t* p, int has_a_scale) {
  if (!p) return 0;
  const mx_linear_problem_t q = as_mxfp8(*p);
  if (!linear_sizes_ok(q) || !linear_supported(q) || p->M == 0) return 0;
  return mx4_plan(*p, has_a_scale != 0).total;
}

extern "C" moe_status_t mx4_linear(const mx4_linear_problem_t* p, const mx_linear_tensors_t* t, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  if (!p || !t) return MOE_ERR_INVALID_ARG;
  const mx_linear_problem_t q = as_mxfp8(*p);
  LinearCall call;
  const moe_status_t v = check_linear(q, *t, call);
  if (v != MOE_OK || p->M == 0) return v;
  const Mx4Plan f = mx4_plan(*p, t->a_scale != nullptr);
  if (f.total > 0 && (!workspace || workspace_bytes < f.total)) return MOE_ERR_WORKSPACE;
  if (f.total > 0 && (uintptr_t)workspace % 256) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;

  const int64_t M = p->M, K = p->K;
  uint8_t* ws = (uint8_t*)workspace;
  const uint8_t* codes = (const uint8_t*)t->a;
  const uint8_t* scales = t->a_scale;
  if (!scales && f.kind != Fc4::kFew) {
    const moe_status_t r = mx4_quantize(t->a, MOE_SRC_BF16, 1, M, K, K, 0, nullptr, nullptr, ws + f.codes,
                                        ws + f.scales, stream);
    if (r != MOE_OK) return r;
    codes = ws + f.codes;
    scales = ws + f.scales;
  }
  if (f.kind == Fc4::kWiden) {
    if (launch_mx4_expand(codes, M * K / 2, ws + f.wide, stream) != hipSuccess) return MOE_ERR_HIP;
    mx_linear_tensors_t u = *t;
    u.a = ws + f.wide;
    u.a_scale = scales;
    return mx_linear(&q, &u, f.rest_bytes ? ws + f.rest : nullptr, f.rest_bytes, stream);
  }
  FcArgs g = linear_args(q, *t, call);
  g.a = codes;
  g.a_scale = scales;
  if (f.kind == Fc4::kFew) {
    if (p->groups > 0) {
      g.group_offsets = t->expert_offsets;
      g.groups = p->groups;
      g.group_rows = (int)M;
      g.max_tiles = f.max_tiles;
    } else {
      g.dense_rows = (int)M;
    }
    g.nchunks = (int)((p->N + kFewCols - 1) / kFewCols);
    return launch_mx4_few(g, !t->a_scale, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  if (p->groups > 0) {
    Tile* tiles = (Tile*)(ws + f.tiles);
    int32_t* ntiles = (int32_t*)(ws + f.ntiles);
    if (launch_group_tiles(t->expert_offsets, p->groups, M, f.rows, tiles, ntiles, stream) != hipSuccess)
      return MOE_ERR_HIP;
    g.tiles = tiles;
    g.num_tiles = ntiles;
    g.max_tiles = f.max_tiles;
  } else {
    g.dense_rows = (int)M;
  }
  g.nchunks = (int)((p->N + kFp4Cols - 1) / kFp4Cols);
  if (f.ksplit > 1) {
    g.ksplit = f.ksplit;
    g.part = (float*)(ws + f.part);
  }
  hipError_t e = launch_linear_fp4(g, f.rows, device_cus(), stream);
  if (e == hipSuccess && f.ksplit > 1) e = launch_linear_join(g, stream);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
