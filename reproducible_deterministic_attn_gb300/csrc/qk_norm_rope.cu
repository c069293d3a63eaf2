// Norm and rotation of queries and keys by one position a token (dash_qk_norm_rope_*).
#include "qk_norm_rope.cuh"

using namespace dash;
using namespace dash::rope;

extern "C" {

dash_status_t dash_qk_norm_rope_fwd(const void* q, const void* k, const float* wq, const float* wk,
                                    const float* cos, const float* sin, const void* positions,
                                    void* q_out, void* k_out, int* status, int B, int S, int Hq,
                                    int Hk, int D, int R, long long P, const long long* q_strides,
                                    const long long* k_strides, long long pos_stride, float eps,
                                    int interleaved, int dtype, int id_bits, cudaStream_t stream) {
  dash_status_t st = check(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides,
                           pos_stride, eps, interleaved, dtype, id_bits);
  if (st != DASH_OK) return st;
  const Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride,
                        eps, interleaved, id_bits);
  return run_fwd<false>(a, q_out, k_out, status, dtype, stream);
}

size_t dash_qk_norm_rope_bwd_workspace_size(int B, int S, int Hq, int Hk, int D) {
  return bwd_workspace_size(B, S, Hq, Hk, D);
}

dash_status_t dash_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                                    const void* k, const float* wq, const float* wk,
                                    const float* cos, const float* sin, const void* positions,
                                    void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                                    size_t workspace_bytes, int B, int S, int Hq, int Hk, int D,
                                    int R, long long P, const long long* q_strides,
                                    const long long* k_strides, const long long* dq_strides,
                                    const long long* dk_strides, long long pos_stride, float eps,
                                    int interleaved, int dtype, int id_bits, cudaStream_t stream) {
  dash_status_t st = check(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides,
                           pos_stride, eps, interleaved, dtype, id_bits);
  if (st != DASH_OK) return st;
  const Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride,
                        eps, interleaved, id_bits);
  return run_bwd<false>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, workspace_bytes, B, dq_strides, dk_strides,
                        dtype, stream);
}

}  // extern "C"
