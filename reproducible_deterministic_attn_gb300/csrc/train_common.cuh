// Device helpers shared by the training-step operators: element conversion, vector access,
// index loads and the report of an index out of range.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dash {
namespace train {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N consecutive elements as one access where N > 1 (the caller guarantees 16-byte alignment
// then; 8 fp32 are two 16-byte accesses).
template <typename T, int N>
struct alignas(N == 1 ? alignof(T) : 16) Vec {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& x) {
  *reinterpret_cast<Vec<T, N>*>(p) = x;
}
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&out)[N]) {
  const Vec<T, N> x = load_vec<T, N>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = to_f32(x.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[N]) {
  Vec<T, N> y;
#pragma unroll
  for (int i = 0; i < N; ++i) y.v[i] = from_f32<T>(x[i]);
  store_vec<T, N>(p, y);
}

// Element i of an int32 or int64 index array.
__device__ __forceinline__ long long load_index(const void* p, long long i, int id_bits) {
  return id_bits == 64 ? __ldg(reinterpret_cast<const long long*>(p) + i)
                       : (long long)__ldg(reinterpret_cast<const int*>(p) + i);
}

// Records an index out of range (the first one of a call wins) in a workspace header.
__device__ __noinline__ inline void report_index(int* header, int site, long long row,
                                                 long long value, long long bound) {
  if (atomicCAS(header + WS_STATUS, 0, kStatusBounds) == 0) {
    header[WS_BH] = (int)row;
    header[WS_QTILE] = site;
    header[WS_EXPECT] = (int)value;
    header[WS_SEEN] = (int)bound;
    __threadfence();
  }
}

}  // namespace train
}  // namespace dash
