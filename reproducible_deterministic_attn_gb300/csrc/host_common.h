// Host-side pieces shared by the library's translation units: the last error's text, the
// tensor-map encoder and small argument checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "dash_attn.h"

namespace dash {

// Text that dash_last_error() returns on this thread.
void set_last_error(const std::string& text);

// cuTensorMapEncodeTiled from the driver, fetched through the runtime (no -lcuda); null
// when the driver has none.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

// Bound on one in-kernel wait (dash_debug_set_sync).
long long sync_timeout_ns();
// Whether the testing hook asks for waits that cannot be satisfied (a skew > 0).
bool sync_withheld();

inline dash_status_t cuda_failed(cudaError_t e, const char* what) {
  set_last_error(std::string(what) + ": " + cudaGetErrorString(e));
  return DASH_ERR_CUDA;
}

inline bool is_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t round_up_to(size_t x, size_t a) { return (x + a - 1) / a * a; }
template <typename T>
inline T ceil_div(T a, T b) { return (a + b - 1) / b; }

// Lets a kernel use `bytes` of dynamic shared memory on the current device (asked of the driver
// once for each kernel and device).
cudaError_t allow_shared(const void* kernel, int bytes);

// Launches a kernel that may start while the kernel before it on `stream` is still running:
// its blocks take their places as that one's leave, and wait for its results with
// grid_wait() before they touch memory. The kernel before must have called grid_next().
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace dash

#define DASH_TRY(call)                                          \
  do {                                                          \
    cudaError_t e_ = (call);                                    \
    if (e_ != cudaSuccess) return dash::cuda_failed(e_, #call); \
  } while (0)
