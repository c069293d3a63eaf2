// Global gradient norm over many tensors and clipping (dash_grad_clip*).
//
// A plan is a device table of pieces of 4096 to 32768 elements. clip_norm walks it with a
// fixed number of blocks: a thread sums the squares of its elements of a piece in fp32 and
// adds the piece's sum to an fp64 total, a block's totals are added by a fixed tree, and the
// last block to finish adds the blocks' totals in order (so the sum's order never depends on
// which block that is). clip_scale then walks the pieces from the end, where the cache still
// holds what the norm read last, and returns at once when nothing has to be written. Both
// are bound by HBM: the norm of 0.5 GB takes 78 us (6.4 TB/s), 2.4 GB clipped into buffers
// 1.09 ms (7.3 GB moved, 6.6 TB/s); four loads of 16 bytes in flight a thread instead of
// eight, and the table read when it is needed: 147 us and 2.0 ms.
#include <algorithm>
#include <exception>
#include <vector>

#include "dash_train.h"
#include "host_common.h"
#include "train_common.cuh"

namespace {

using namespace dash;
using namespace dash::train;

constexpr int kMaxPiece = 32768, kMinPiece = 4096;
constexpr int kThreads = 512;
constexpr int kAhead = 8;                // loads of 16 bytes a thread has in flight
constexpr int kBlocks = 608;             // fixes the order of the sum: not the SM count
constexpr unsigned long long kMagic = 0x64617368636c6970ull;

struct Piece {
  const void* grad;
  void* out;
  int count, dtype;
};
static_assert(sizeof(Piece) == 24, "table layout");

struct Header {
  unsigned long long magic;
  long long pieces;
  int blocks;                            // that share the sum: min(pieces, kBlocks)
  int all_in_place;
  unsigned done;                         // blocks that have left their total; ends at 0
  double norm;
  double totals[kBlocks];
};
constexpr size_t kTableOff = (sizeof(Header) + 255) / 256 * 256;

// Whether this is a plan whose table lies within the caller's buffer (`capacity` pieces) and
// whose blocks the launch has. No other plan's table is read.
__device__ __forceinline__ bool plan_fits(const Header* h, long long capacity) {
  return h->magic == kMagic && h->pieces >= 0 && h->pieces <= capacity && h->blocks >= 1 &&
         h->blocks <= (int)gridDim.x;
}

// The elements' bits, ORed into one word.
template <typename T, int N>
__device__ __forceinline__ void or_bits(uint32_t& any, const Vec<T, N>& v) {
  if constexpr (N == 1) {
    any |= sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(&v.w) : *reinterpret_cast<const uint16_t*>(&v.w);
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 4); ++i) any |= v.w[i];
  }
}

// Sum of squares of this thread's elements of a piece. 32 bits hold the sum unless it
// overflows or is so small that squares may have vanished; then the elements are scaled by
// the power of two that brings their largest to [1/2, 1). Elements that are all zero, as whole
// rows of a table's gradient are, are known by their bits: read a second time they made the norm
// of four gradients of 65536 x 2048 bf16 take 182 us with a fifth of the rows present and 343
// with none, where dense ones take 160 (now 158 each).
template <typename T, int VEC>
__device__ __forceinline__ double squares(const T* x, int count) {
  constexpr int kStep = kThreads * VEC;
  float s[4] = {};
  uint32_t any = 0;
  const int whole = count / VEC * VEC;
  int i = threadIdx.x * VEC;
#pragma unroll 1
  for (; i + (kAhead - 1) * kStep < whole; i += kAhead * kStep) {
    Vec<T, VEC> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = load_vec<T, VEC>(x + i + u * kStep);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float f[VEC];
      or_bits<T, VEC>(any, v[u]);
      unpack<T, VEC>(v[u], f);
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[k & 3] = fmaf(f[k], f[k], s[k & 3]);
    }
  }
#pragma unroll 1
  for (; i < whole; i += kStep) {
    float f[VEC];
    const Vec<T, VEC> v = load_vec<T, VEC>(x + i);
    or_bits<T, VEC>(any, v);
    unpack<T, VEC>(v, f);
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k & 3] = fmaf(f[k], f[k], s[k & 3]);
  }
#pragma unroll 1
  for (int j = whole + threadIdx.x; j < count; j += kThreads) {
    const Vec<T, 1> v = load_vec<T, 1>(x + j);
    or_bits<T, 1>(any, v);
    const float f = to_f32(v.w);
    s[0] = fmaf(f, f, s[0]);
  }
  const float t = (s[0] + s[1]) + (s[2] + s[3]);
  if (t > 0x1p-90f && t < 0x1p126f) return (double)t;
  if ((any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return 0.0;
  // the thread's elements once more: the same ones as above
  auto each = [&](auto f) {
#pragma unroll 1
    for (int j = threadIdx.x * VEC; j < whole; j += kStep) {
      float z[VEC];
      load_f32<T, VEC>(x + j, z);
#pragma unroll
      for (int k = 0; k < VEC; ++k) f(z[k]);
    }
#pragma unroll 1
    for (int j = whole + threadIdx.x; j < count; j += kThreads) f(to_f32(x[j]));
  };
  float big = 0.f;
  bool nan = false;
  each([&](float f) {
    nan |= f != f;
    big = fmaxf(big, fabsf(f));
  });
  if (nan) return (double)NAN;
  if (isinf(big)) return (double)INFINITY;
  int e;
  frexpf(big, &e);
  float p = 0.f;
  each([&](float f) {
    f = ldexpf(f, -e);
    p = fmaf(f, f, p);
  });
  return ldexp((double)p, 2 * e);
}

template <typename T>
__device__ __forceinline__ double squares_of(const Piece& pc) {
  constexpr int W = 16 / sizeof(T);
  const T* x = (const T*)pc.grad;
  return ((uintptr_t)x & 15) == 0 ? squares<T, W>(x, pc.count) : squares<T, 1>(x, pc.count);
}

__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) t += shared[w];
  return t;                              // thread 0's
}

__global__ void __launch_bounds__(kThreads, 2) clip_norm_kernel(Header* h, const Piece* table,
                                                                 long long capacity, float* norm) {
  __shared__ double shared[kThreads / 32];
  __shared__ bool last;
  grid_next();
  if (!plan_fits(h, capacity)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = NAN;
    return;
  }
  const long long pieces = h->pieces;
  const int blocks = h->blocks;
  if (blockIdx.x >= blocks) return;
  double sum = 0.0;
  Piece next = {};
  if (blockIdx.x < pieces) next = table[blockIdx.x];
  for (long long i = blockIdx.x; i < pieces; i += blocks) {
    const Piece pc = next;
    if (i + blocks < pieces) next = table[i + blocks];
    sum += pc.dtype == DASH_BF16   ? squares_of<__nv_bfloat16>(pc)
           : pc.dtype == DASH_FP16 ? squares_of<__half>(pc)
                                   : squares_of<float>(pc);
  }
  const double mine = block_sum(sum, shared);
  if (threadIdx.x == 0) {
    h->totals[blockIdx.x] = mine;
    __threadfence();
    last = atomicAdd(&h->done, 1u) == blocks - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < blocks; i += kThreads) v += __ldcg(&h->totals[i]);
  const double all = block_sum(v, shared);
  if (threadIdx.x == 0) {
    const double n = sqrt(all);
    h->norm = n;
    *norm = (float)n;
    h->done = 0;
  }
}

// The factor max_norm / norm as a product, the second one a power of two: 1, unless a single
// fp32 would be below the normal range and lose bits.
struct Factor {
  float f, g;
  __device__ __forceinline__ float operator()(float x) const { return x * f * g; }
};
__device__ __forceinline__ Factor factor(double x) {
  if (x >= 0x1p-126 || x == 0.0) return {(float)x, 1.f};
  int e;
  frexp(x, &e);
  const double g = ldexp(1.0, max(e, -149));
  return {(float)(x / g), (float)g};
}

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> scaled(const Vec<T, VEC>& v, Factor f, bool copy) {
  float z[VEC];
  unpack<T, VEC>(v, z);
#pragma unroll
  for (int k = 0; k < VEC; ++k) z[k] = f(z[k]);
  return copy ? v : pack<T, VEC>(z);
}

template <typename T, int VEC>
__device__ __forceinline__ void scale_piece(const T* x, T* y, int count, Factor f, bool copy) {
  constexpr int kStep = kThreads * VEC;
  const int whole = count / VEC * VEC;
  int i = threadIdx.x * VEC;
#pragma unroll 1
  for (; i + (kAhead - 1) * kStep < whole; i += kAhead * kStep) {
    Vec<T, VEC> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = load_vec<T, VEC>(x + i + u * kStep);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) store_vec<T, VEC>(y + i + u * kStep, scaled<T, VEC>(v[u], f, copy));
  }
#pragma unroll 1
  for (; i < whole; i += kStep) store_vec<T, VEC>(y + i, scaled<T, VEC>(load_vec<T, VEC>(x + i), f, copy));
#pragma unroll 1
  for (int j = whole + threadIdx.x; j < count; j += kThreads)
    y[j] = copy ? x[j] : from_f32<T>(f(to_f32(x[j])));
}

template <typename T>
__device__ __forceinline__ void scale_of(const Piece& pc, Factor f, bool copy) {
  constexpr int W = 16 / sizeof(T);
  const T* x = (const T*)pc.grad;
  T* y = (T*)pc.out;
  if ((((uintptr_t)x | (uintptr_t)y) & 15) == 0) scale_piece<T, W>(x, y, pc.count, f, copy);
  else scale_piece<T, 1>(x, y, pc.count, f, copy);
}

__global__ void __launch_bounds__(kThreads, 2) clip_scale_kernel(const Header* h, const Piece* table,
                                                                  long long capacity, float max_norm) {
  // the table and its header's constants are the plan's, not the kernel's before
  const bool ok = plan_fits(h, capacity);
  const long long first = ok ? h->pieces - 1 - blockIdx.x : -1;
  Piece next = {};
  if (first >= 0) next = table[first];
  grid_wait();
  if (!ok) return;
  const double n = h->norm;
  const bool copy = !(n > (double)max_norm) || isinf((float)n);   // as the caller's norm says
  if (copy && h->all_in_place) return;
  const Factor f = factor(copy ? 1.0 : (double)max_norm / n);
  for (long long i = first; i >= 0; i -= gridDim.x) {
    const Piece pc = next;
    if (i >= gridDim.x) next = table[i - gridDim.x];
    if (copy && pc.out == pc.grad) continue;
    if (pc.dtype == DASH_BF16) scale_of<__nv_bfloat16>(pc, f, copy);
    else if (pc.dtype == DASH_FP16) scale_of<__half>(pc, f, copy);
    else scale_of<float>(pc, f, copy);
  }
}

// Checks a list; its number of pieces and their size, or a status. Pieces are halved while
// there are too few for all blocks, so that few elements still spread over the chip.
dash_status_t cut(const dash_clip_tensor_t* t, int n, long long* pieces, int* piece) {
  if (!t || n < 1) return DASH_ERR_INVALID_ARG;
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel < 0 || t[i].dtype < DASH_BF16 || t[i].dtype > DASH_FP32) return DASH_ERR_INVALID_ARG;
    const uintptr_t e = t[i].dtype == DASH_FP32 ? 4 : 2;
    if (t[i].numel > 0 && (!t[i].grad || !t[i].out)) return DASH_ERR_INVALID_ARG;
    if (!is_aligned(t[i].grad, e) || !is_aligned(t[i].out, e)) return DASH_ERR_INVALID_ARG;
    if (t[i].numel > (1ll << 45) || total > (1ll << 45)) return DASH_ERR_UNSUPPORTED;
    total += t[i].numel;
  }
  *piece = kMaxPiece;
  while (*piece > kMinPiece && total / *piece < kBlocks) *piece /= 2;
  *pieces = 0;
  for (int i = 0; i < n; ++i) *pieces += ceil_div<long long>(t[i].numel, *piece);
  return *pieces > (1ll << 31) ? DASH_ERR_UNSUPPORTED : DASH_OK;
}

}  // namespace

extern "C" {

size_t dash_grad_clip_plan_size(const dash_clip_tensor_t* tensors, int n) {
  long long pieces;
  int piece;
  return cut(tensors, n, &pieces, &piece) != DASH_OK ? 0 : kTableOff + round_up_to((size_t)pieces * sizeof(Piece), 256);
}

dash_status_t dash_grad_clip_plan(const dash_clip_tensor_t* tensors, int n, void* plan,
                                  size_t plan_bytes, cudaStream_t stream) {
  long long pieces;
  int piece;
  const dash_status_t st = cut(tensors, n, &pieces, &piece);
  if (st != DASH_OK) return st;
  if (!plan || !is_aligned(plan, 256)) return DASH_ERR_INVALID_ARG;
  if (plan_bytes < kTableOff + (size_t)pieces * sizeof(Piece)) return DASH_ERR_WORKSPACE_TOO_SMALL;
  try {
    std::vector<Piece> table;
    table.reserve(pieces);
    Header h = {};
    h.magic = kMagic;
    h.pieces = pieces;
    h.blocks = (int)std::min<long long>(kBlocks, std::max<long long>(pieces, 1));
    h.all_in_place = 1;
    for (int i = 0; i < n; ++i) {
      const size_t e = tensors[i].dtype == DASH_FP32 ? 4 : 2;
      if (tensors[i].numel > 0 && tensors[i].grad != tensors[i].out) h.all_in_place = 0;
      for (long long at = 0; at < tensors[i].numel; at += piece)
        table.push_back({(const char*)tensors[i].grad + at * e, (char*)tensors[i].out + at * e,
                         (int)std::min<long long>(piece, tensors[i].numel - at), tensors[i].dtype});
    }
    DASH_TRY(cudaMemcpyAsync(plan, &h, sizeof(h), cudaMemcpyHostToDevice, stream));
    if (pieces > 0)
      DASH_TRY(cudaMemcpyAsync((char*)plan + kTableOff, table.data(), table.size() * sizeof(Piece),
                               cudaMemcpyHostToDevice, stream));
    DASH_TRY(cudaStreamSynchronize(stream));
  } catch (const std::exception& e) {
    set_last_error(std::string("dash_grad_clip_plan: ") + e.what());
    return DASH_ERR_UNSUPPORTED;
  }
  return DASH_OK;
}

dash_status_t dash_grad_clip(void* plan, size_t plan_bytes, float max_norm, float* norm, cudaStream_t stream) {
  if (!plan || !norm || !is_aligned(plan, 256) || !is_aligned(norm, 4)) return DASH_ERR_INVALID_ARG;
  if (plan_bytes < kTableOff) return DASH_ERR_WORKSPACE_TOO_SMALL;
  if (!(max_norm >= 0.f)) return DASH_ERR_INVALID_ARG;
  Header* h = (Header*)plan;
  const Piece* table = (const Piece*)((char*)plan + kTableOff);
  // no more blocks than the table can hold pieces for (the header has the exact number)
  const long long capacity = (long long)((plan_bytes - kTableOff) / sizeof(Piece));
  const int grid = (int)std::max<long long>(1, std::min<long long>(kBlocks, capacity));
  clip_norm_kernel<<<grid, kThreads, 0, stream>>>(h, table, capacity, norm);
  DASH_TRY(cudaGetLastError());
  DASH_TRY(launch_after(clip_scale_kernel, dim3(grid), kThreads, 0, stream, h, table, capacity, max_norm));
  return DASH_OK;
}

}  // extern "C"
