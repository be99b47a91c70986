// mx4_linear: the matrix product with MXFP4 operands on both sides and mx_linear's
// epilogue (mxfp6-sm120 page, table of paths, "Dense" row, and "Execution model";
// TokenSpeed SiTU page, "Supported contract": MxE2m1).
//
// Every E2M1 value is an E4M3 value, so E2M1 activations are also MXFP8 activations
// with the same scales: their codes are widened in the workspace and multiplied by
// mx_linear's kernels.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "linear_plan.h"

namespace moe_mx {

namespace {

// Workspace of a call
struct Plan4 {
  size_t codes, scales;  // E2M1 codes and scales of bf16 rows
  size_t wide;           // their E4M3 codes
  size_t rest, total;    // mx_linear's own
};

mx_linear_problem_t as_mxfp8(const mx4_linear_problem_t& p) {
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

Plan4 plan4(const mx4_linear_problem_t& p, bool has_a_scale) {
  const mx_linear_problem_t q = as_mxfp8(p);
  Plan4 f = {};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = align_up(o + bytes, 256);
    return r;
  };
  if (!has_a_scale) {
    f.codes = take((size_t)(p.M * p.K / 2));
    f.scales = take((size_t)(p.M * p.K / 32));
  }
  f.wide = take((size_t)(p.M * p.K));
  f.rest = o;
  f.total = o + mx_linear_workspace_bytes(&q, 1);
  return f;
}

}  // namespace

}  // namespace moe_mx

using namespace moe_mx;

extern "C" size_t mx4_linear_workspace_bytes(const mx4_linear_problem_t* p, int has_a_scale) {
  if (!p) return 0;
  const mx_linear_problem_t q = as_mxfp8(*p);
  if (!linear_sizes_ok(q) || !linear_supported(q) || p->M == 0) return 0;
  return plan4(*p, has_a_scale != 0).total;
}

extern "C" moe_status_t mx4_linear(const mx4_linear_problem_t* p, const mx_linear_tensors_t* t, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  if (!p || !t) return MOE_ERR_INVALID_ARG;
  const mx_linear_problem_t q = as_mxfp8(*p);
  if (!linear_sizes_ok(q)) return MOE_ERR_INVALID_ARG;
  if (!linear_supported(q)) return MOE_ERR_UNSUPPORTED;
  if (p->M == 0) return MOE_OK;
  if (!t->a || (uintptr_t)t->a % 16 || (uintptr_t)t->a_scale % 16) return MOE_ERR_INVALID_ARG;
  const Plan4 f = plan4(*p, t->a_scale != nullptr);
  if (!workspace || workspace_bytes < f.total) return MOE_ERR_WORKSPACE;
  if ((uintptr_t)workspace % 256) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_arch();
  if (st != MOE_OK) return st;
  uint8_t* ws = (uint8_t*)workspace;
  const uint8_t* codes = (const uint8_t*)t->a;
  const uint8_t* scales = t->a_scale;
  if (!scales) {
    const moe_status_t r = mx4_quantize(t->a, MOE_SRC_BF16, 1, p->M, p->K, p->K, 0, nullptr, nullptr, ws + f.codes,
                                        ws + f.scales, stream);
    if (r != MOE_OK) return r;
    codes = ws + f.codes;
    scales = ws + f.scales;
  }
  if (launch_mx4_expand(codes, p->M * p->K / 2, ws + f.wide, stream) != hipSuccess) return MOE_ERR_HIP;
  mx_linear_tensors_t u = *t;
  u.a = ws + f.wide;
  u.a_scale = scales;
  return mx_linear(&q, &u, ws + f.rest, f.total - f.rest, stream);
}
