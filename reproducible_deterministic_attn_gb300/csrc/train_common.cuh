// Device helpers shared by the training-step operators: element conversion, vector access,
// index loads and the report of an index out of range.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dash {
namespace train {

// Kernels of one call overlap their starts: each lets the next one's blocks take their places
// once all of its own run (grid_next), and each but the first waits for the memory of those
// before it (grid_wait) before it reads or writes any.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// N consecutive elements as they lie in memory, in whole 32-bit words where N > 1 (so that 16-bit
// elements stay packed two to a register until they are used), accessed 16 bytes at a time
// (the caller guarantees that alignment then).
template <typename T, int N>
struct Vec {
  static_assert(N * sizeof(T) % 16 == 0, "whole 16-byte pieces");
  uint32_t w[N * sizeof(T) / 4];
};
template <typename T>
struct Vec<T, 1> {
  T w;
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
  Vec<T, N> x;
  if constexpr (N == 1) {
    x.w = *p;
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      x.w[4 * i] = v.x;
      x.w[4 * i + 1] = v.y;
      x.w[4 * i + 2] = v.z;
      x.w[4 * i + 3] = v.w;
    }
  }
  return x;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& x) {
  if constexpr (N == 1) {
    *p = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(x.w[4 * i], x.w[4 * i + 1], x.w[4 * i + 2], x.w[4 * i + 3]);
  }
}

// The two 16-bit elements of a word, the lower address first.
template <typename T>
__device__ __forceinline__ float2 halves(uint32_t w);
template <>
__device__ __forceinline__ float2 halves<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 halves<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_halves(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_halves<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack_halves<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int N>
__device__ __forceinline__ void unpack(const Vec<T, N>& x, float (&out)[N]) {
  if constexpr (N == 1) {
    out[0] = to_f32(x.w);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __uint_as_float(x.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 f = halves<T>(x.w[i / 2]);
      out[i] = f.x;
      out[i + 1] = f.y;
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> pack(const float (&x)[N]) {
  Vec<T, N> y;
  if constexpr (N == 1) {
    y.w = from_f32<T>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) y.w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) y.w[i / 2] = pack_halves<T>(x[i], x[i + 1]);
  }
  return y;
}

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&out)[N]) {
  unpack<T, N>(load_vec<T, N>(p), out);
}
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[N]) {
  store_vec<T, N>(p, pack<T, N>(x));
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
