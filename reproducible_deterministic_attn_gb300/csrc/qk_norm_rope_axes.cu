// Norm and rotation of queries and keys by positions with several axes (dash_qk_norm_rope_axes_*).
#include "qk_norm_rope.cuh"

using namespace dash;
using namespace dash::rope;

namespace {

// The pairs' axes, 2 bits each.
dash_status_t set_axes(Args* a, const void* positions, const int* sections, int axes, long long axis_stride,
                       long long P) {
  if (!sections || axes < 1 || axes > kMaxAxes || axis_stride < 0) return DASH_ERR_INVALID_ARG;
  if (a->tokens > 0 && !positions) return DASH_ERR_INVALID_ARG;
  if (axis_stride > (1ll << 40) || P >= (1ll << 31)) return DASH_ERR_UNSUPPORTED;
  int i = 0;
  for (int x = 0; x < axes; ++x) {
    if (sections[x] < 0 || sections[x] > a->R / 2 - i) return DASH_ERR_INVALID_ARG;
    for (int n = 0; n < sections[x]; ++n, ++i) a->pair_axis[i >> 4] |= (uint32_t)x << (2 * (i & 15));
  }
  if (i != a->R / 2) return DASH_ERR_INVALID_ARG;
  a->axes = axes;
  a->axis_stride = axis_stride;
  return DASH_OK;
}

}  // namespace

extern "C" {

dash_status_t dash_qk_norm_rope_axes_fwd(const void* q, const void* k, const float* wq, const float* wk,
                                         const float* cos, const float* sin, const void* positions, void* q_out,
                                         void* k_out, int* status, int B, int S, int Hq, int Hk, int D, int R,
                                         long long P, const long long* q_strides, const long long* k_strides,
                                         const int* sections, int axes, long long axis_stride, long long pos_stride,
                                         float eps, int interleaved, int dtype, int id_bits, cudaStream_t stream) {
  dash_status_t st = check(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides,
                           pos_stride, eps, interleaved, dtype, id_bits);
  if (st != DASH_OK) return st;
  Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride, eps,
                  interleaved, id_bits);
  st = set_axes(&a, positions, sections, axes, axis_stride, P);
  if (st != DASH_OK) return st;
  return run_fwd<true>(a, q_out, k_out, status, dtype, stream);
}

dash_status_t dash_qk_norm_rope_axes_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                                         const float* wq, const float* wk, const float* cos, const float* sin,
                                         const void* positions, void* dq, void* dk, float* dwq, float* dwk,
                                         void* workspace, size_t workspace_bytes, int B, int S, int Hq, int Hk,
                                         int D, int R, long long P, const long long* q_strides,
                                         const long long* k_strides, const long long* dq_strides,
                                         const long long* dk_strides, const int* sections, int axes,
                                         long long axis_stride, long long pos_stride, float eps, int interleaved,
                                         int dtype, int id_bits, cudaStream_t stream) {
  dash_status_t st = check(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides,
                           pos_stride, eps, interleaved, dtype, id_bits);
  if (st != DASH_OK) return st;
  Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride, eps,
                  interleaved, id_bits);
  st = set_axes(&a, positions, sections, axes, axis_stride, P);
  if (st != DASH_OK) return st;
  return run_bwd<true>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, workspace_bytes, B, dq_strides, dk_strides,
                       dtype, stream);
}

}  // extern "C"
