// Norm of queries and keys per head with the rotation in the same pass (dash_qk_norm_rope_*).
//
// A head's D values lie in L = D / 8 lanes of a warp (rounded up to a power of two), 8 values
// and one 16-byte access a lane (two in fp32), so the mean of squares is a shuffle tree and
// the rotation's partner values come from the lane R / 16 away, or, where R / 2 is no
// multiple of 8, from a second read of the row (which hits L1). A warp keeps one token's
// angles and weights in registers over several heads. Both directions read and write every
// value once: bound by HBM.
#include <algorithm>

#include "dash_train.h"
#include "host_common.h"
#include "train_common.cuh"

namespace {

using namespace dash;
using namespace dash::train;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 256;
// Blocks that share the rows. The backward's number fixes how dw's sum is split, so it is a
// constant and not the device's SM count: one block for each that 152 SMs hold.
constexpr int kFwdBlocks = 608 * 2;
constexpr int kBwdBlocks = 304;
static_assert(2 * (kBwdBlocks + 1) <= 1024, "dw_join looks at all blocks at once");

struct Side {                       // queries or keys
  const void* x;
  const float* w;
  const void* dout;                 // backward: contiguous gradient of the output
  void* out;                        // forward: contiguous output; backward: dx
  long long sb, ss, sh;             // strides of x
  long long ob, os, oh;             // strides of out
  float* dw;
  float* part;                      // backward: [blocks][D]
  int* bad;                         // backward: [blocks], lowest token whose position is out of range
  int H;
  int blocks;                       // of the grid
};

struct Args {
  Side side[2];
  const float *cos, *sin;
  const void* pos;
  long long pos_stride, P;
  int id_bits;
  int tokens, S, D, R;
  float eps;
  int* header;                      // backward: workspace header
  int* status;                      // forward: optional status word
};

// cos and sin of the pairs that a lane's 8 columns belong to.
template <bool IL>
struct Angles {
  float c[IL ? 4 : 8], s[IL ? 4 : 8];
};

// Position of a token, out of range or not.
__device__ __forceinline__ long long load_position(const Args& a, int token) {
  const int b = token / a.S, s = token - b * a.S;
  return a.pos ? load_index(a.pos, b * a.pos_stride + s, a.id_bits) : (long long)s;
}

constexpr int kNoToken = 0x7fffffff;

__device__ __forceinline__ void four(const float* p, float* v) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}

// FAST: a lane's columns are all rotated or none, and its angles are whole 16-byte pieces.
template <bool IL, bool FAST>
__device__ __forceinline__ void load_angles(const Args& a, long long p, int col, Angles<IL>& g) {
  const int half = a.R >> 1;
  constexpr int N = IL ? 4 : 8;
  if constexpr (FAST) {
    if (col < a.R && p >= 0) {
      const long long at = p * half + (IL ? col >> 1 : col < half ? col : col - half);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        four(a.cos + at + i, g.c + i);
        four(a.sin + at + i, g.s + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        g.c[i] = 1.f;      // a position out of range makes the norm NaN
        g.s[i] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = IL ? (col >> 1) + i : (col + i < half ? col + i : col + i - half);
      const bool in = (IL ? col + 2 * i : col + i) < a.R && p >= 0;
      g.c[i] = in ? __ldg(a.cos + p * half + j) : 1.f;
      g.s[i] = in ? __ldg(a.sin + p * half + j) : 0.f;
    }
  }
}

// Rotates the 8 values y of columns col.. (sign +1) or applies the transpose (sign -1).
// Half-split pairs, FAST: they lie whole lanes apart (R / 2 a multiple of 8); else `partner(c)`
// gives the value of column c.
template <bool IL, bool FAST, typename F>
__device__ __forceinline__ void rotate(const Args& a, const Angles<IL>& g, int col, float sign, float (&y)[8],
                                       F partner) {
  const int half = a.R >> 1;
  if (IL) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = y[2 * i], v = y[2 * i + 1], s = sign * g.s[i];
      y[2 * i] = u * g.c[i] - v * s;
      y[2 * i + 1] = v * g.c[i] + u * s;
    }
  } else if (FAST) {
    const int d = half >> 3;
    const int lane = threadIdx.x & 31;
    const bool lo = col < half;
    const int src = lo ? lane + d : lane - d;
    const float sg = lo ? -sign : sign;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, y[i], src);
      if (col < a.R) y[i] = y[i] * g.c[i] + o * (sg * g.s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col + i;
      if (c < a.R) {
        const float o = partner(c < half ? c + half : c - half);
        y[i] = y[i] * g.c[i] + (c < half ? -sign : sign) * (o * g.s[i]);
      }
    }
  }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void load_weights(const float* w, int col, bool in, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.f;
  if (w && in) {
    four(w + col, v);
    four(w + col + 4, v + 4);
  }
}

// Forward. A warp walks over items of one token and U * 32 / L heads, the grid's warps apart.
// The next item's position is fetched an item ahead, so that the angles' loads, which need
// it, start together with the data's.
template <typename T, int L, bool IL, bool FAST, int U>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args a) {
  constexpr int RW = 32 / L;                       // heads a warp handles at once
  const int which = blockIdx.x >= a.side[0].blocks;
  const Side& sd = a.side[which];
  const int lane = threadIdx.x & 31, sub = lane / L, col = (lane % L) * 8;
  const unsigned groups = (unsigned)(sd.H + U * RW - 1) / (U * RW), items = (unsigned)a.tokens * groups;
  const unsigned step = (unsigned)sd.blocks * kWarps;
  unsigned item = (blockIdx.x - (which ? a.side[0].blocks : 0)) * kWarps + (threadIdx.x >> 5);
  if (item >= items) return;
  const bool in = col < a.D;
  const float inv_d = 1.f / a.D;
  float w[8];
  load_weights(sd.w, col, in, w);
  long long next_p = load_position(a, (int)(item / groups));
  for (; item < items; item += step) {
    const int token = (int)(item / groups), h0 = (int)(item % groups) * U * RW + sub;
    const int b = token / a.S, s = token - b * a.S;
    const T* x = (const T*)sd.x + b * sd.sb + s * sd.ss;
    T* out = (T*)sd.out + b * sd.ob + s * sd.os;
    Vec<T, 8> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RW;
      raw[u] = {};
      if (in && h < sd.H) raw[u] = load_vec<T, 8>(x + h * sd.sh + col);
    }
    long long p = next_p;
    if (p < 0 || p >= a.P) {
      p = -1;
      if (a.status) *a.status = kStatusBounds;
    }
    Angles<IL> g;
    load_angles<IL, FAST>(a, p, col, g);
    if (items - item > step) next_p = load_position(a, (int)((item + step) / groups));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RW;
      const bool live = in && h < sd.H;
      float y[8], q = 0.f;
      unpack<T, 8>(raw[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(y[i], y[i], q);
      const float r = p < 0 ? NAN : rsqrtf(lanes_sum<L>(q) * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
      const T* row = x + (long long)h * sd.sh;
      rotate<IL, FAST>(a, g, col, 1.f, y, [&](int c) {
        return live ? to_f32(row[c]) * r * (sd.w ? __ldg(sd.w + c) : 1.f) : 0.f;
      });
      if (live) store_f32<T, 8>(out + h * sd.oh + col, y);
    }
  }
}

// Backward. A warp walks over (token, head group) items, `blocks` blocks apart, and keeps its
// columns' part of dw in registers; the block's warps are added in order.
template <typename T, int L, bool IL, bool FAST, int U>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args a) {
  constexpr int RW = 32 / L;
  __shared__ float dws[kWarps][kMaxD];
  __shared__ int bad;
  grid_next();
  if (threadIdx.x == 0) bad = kNoToken;
  __syncthreads();
  const int which = blockIdx.x >= a.side[0].blocks;
  const Side& sd = a.side[which];
  const int block = blockIdx.x - (which ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L, col = (lane % L) * 8;
  const unsigned groups = (unsigned)(sd.H + U * RW - 1) / (U * RW), items = (unsigned)a.tokens * groups;
  const unsigned step = (unsigned)sd.blocks * kWarps;
  const bool in = col < a.D;
  const float inv_d = 1.f / a.D;
  float w[8], dw[8] = {};
  load_weights(sd.w, col, in, w);
  unsigned item = (unsigned)block * kWarps + warp;
  long long next_p = item < items ? load_position(a, (int)(item / groups)) : 0;
  for (; item < items; item += step) {
    const int token = (int)(item / groups), h0 = (int)(item % groups) * U * RW + sub;
    const int b = token / a.S, s = token - b * a.S;
    const T* x = (const T*)sd.x + b * sd.sb + s * sd.ss;
    const T* d = (const T*)sd.dout + (long long)token * sd.H * a.D;
    T* out = (T*)sd.out + b * sd.ob + s * sd.os;
    Vec<T, 8> rx[U], rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RW;
      rx[u] = rd[u] = {};
      if (in && h < sd.H) {
        rx[u] = load_vec<T, 8>(x + h * sd.sh + col);
        rd[u] = load_vec<T, 8>(d + (long long)h * a.D + col);
      }
    }
    long long p = next_p;
    if (p < 0 || p >= a.P) {
      p = -1;
      if (lane == 0) atomicMin(&bad, token);
    }
    Angles<IL> g;
    load_angles<IL, FAST>(a, p, col, g);
    if (items - item > step) next_p = load_position(a, (int)((item + step) / groups));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RW;
      const bool live = in && h < sd.H;
      float n[8], dy[8], q = 0.f;
      unpack<T, 8>(rx[u], n);
      unpack<T, 8>(rd[u], dy);
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(n[i], n[i], q);
      const float r = p < 0 ? NAN : rsqrtf(lanes_sum<L>(q) * inv_d + a.eps);
      rotate<IL, FAST>(a, g, col, -1.f, dy, [&](int c) {
        return live ? to_f32(d[(long long)h * a.D + c]) : 0.f;
      });
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] *= r;
        if (live) dw[i] = fmaf(dy[i], n[i], dw[i]);
        dy[i] *= w[i];
        dot = fmaf(dy[i], n[i], dot);
      }
      dot = lanes_sum<L>(dot) * inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) dy[i] = r * (dy[i] - n[i] * dot);
      if (live) store_f32<T, 8>(out + h * sd.oh + col, dy);
    }
  }
  // heads of the warp, then warps, in order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
    if (sub == 0 && in) dws[warp][col + i] = dw[i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    float t = 0.f;
    for (int k = 0; k < kWarps; ++k) t += dws[k][c];
    sd.part[(long long)block * a.D + c] = t;
  }
  if (threadIdx.x == 0) sd.bad[block] = bad;
}

// dw = the blocks' parts, added in order: 32 groups of consecutive blocks, then the groups.
// One block for each 32 columns of one tensor; the first also writes the call's status.
__global__ void __launch_bounds__(1024) dw_join_kernel(const Args a) {
  __shared__ float sums[32][33];
  __shared__ int first;
  grid_wait();
  const Side& sd = a.side[blockIdx.x];
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) first = kNoToken;
    __syncthreads();
    const int n = a.side[0].blocks, b = threadIdx.x;      // at most 1024 blocks
    if (b < n + a.side[1].blocks) {
      const int t = b < n ? a.side[0].bad[b] : a.side[1].bad[b - n];
      if (t != kNoToken) atomicMin(&first, t);
    }
    __syncthreads();
    if (threadIdx.x < kWsHeaderBytes / 4) {
      int v = 0;
      if (first != kNoToken) {
        if (threadIdx.x == WS_STATUS) v = kStatusBounds;
        if (threadIdx.x == WS_BH) v = first;
        if (threadIdx.x == WS_QTILE) v = CHK_POSITION;
        if (threadIdx.x == WS_EXPECT) v = (int)load_position(a, first);
        if (threadIdx.x == WS_SEEN) v = (int)a.P;
      }
      a.header[threadIdx.x] = v;
    }
  }
  if (!sd.dw) return;
  const int x = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.y * 32 + x;
  const int per = (sd.blocks + 31) / 32;
  const int end = min(sd.blocks, (g + 1) * per);
  float t = 0.f;
  if (c < a.D)
#pragma unroll 8
    for (int k = g * per; k < end; ++k) t += sd.part[(long long)k * a.D + c];
  sums[g][x] = t;
  __syncthreads();
  if (g == 0 && c < a.D) {
    for (int k = 1; k < 32; ++k) t += sums[k][x];
    sd.dw[c] = t;
  }
}

// ---- host ---------------------------------------------------------------------------------

template <typename T, int L, bool IL, bool FAST>
dash_status_t launch(Args a, bool bwd, cudaStream_t stream) {
  constexpr int RW = 32 / L;
  constexpr int U = sizeof(T) == 4 ? 2 : 4;
  // heads in flight a warp: U when that leaves every warp of the chip (about 10^4) an item,
  // else one, which spreads few tokens over more warps
  const long long rows = (long long)a.tokens * (a.side[0].H + a.side[1].H);
  const bool many = rows / (U * RW) >= 9728;
  const int per = many ? U * RW : RW;
  // each tensor's share of the blocks goes by its heads
  const int H = a.side[0].H + a.side[1].H, most = bwd ? kBwdBlocks : kFwdBlocks;
  for (int i = 0; i < 2; ++i) {
    const long long items = (long long)a.tokens * ceil_div(a.side[i].H, per);
    const long long share = H > 0 ? std::max<long long>(1, ((long long)most * a.side[i].H + H / 2) / H) : 0;
    a.side[i].blocks = (int)std::min<long long>(ceil_div<long long>(items, kWarps), share);
  }
  const unsigned grid = a.side[0].blocks + a.side[1].blocks;
  if (grid > 0) {
    if (bwd) {
      if (many) bwd_kernel<T, L, IL, FAST, U><<<grid, kThreads, 0, stream>>>(a);
      else bwd_kernel<T, L, IL, FAST, 1><<<grid, kThreads, 0, stream>>>(a);
    } else {
      if (many) fwd_kernel<T, L, IL, FAST, U><<<grid, kThreads, 0, stream>>>(a);
      else fwd_kernel<T, L, IL, FAST, 1><<<grid, kThreads, 0, stream>>>(a);
    }
    DASH_TRY(cudaGetLastError());
  }
  if (bwd) DASH_TRY(launch_after(dw_join_kernel, dim3(2, ceil_div(a.D, 32)), 1024, 0, stream, a));
  return DASH_OK;
}

template <typename T, int L>
dash_status_t by_pairs(const Args& a, bool bwd, bool interleaved, cudaStream_t stream) {
  if (interleaved)
    return a.R % 8 == 0 ? launch<T, L, true, true>(a, bwd, stream) : launch<T, L, true, false>(a, bwd, stream);
  if ((a.R / 2) % 8 == 0) return launch<T, L, false, true>(a, bwd, stream);
  return launch<T, L, false, false>(a, bwd, stream);
}

template <typename T>
dash_status_t by_lanes(const Args& a, bool bwd, bool interleaved, cudaStream_t stream) {
  const int lanes = a.D / 8;
  if (lanes <= 8) return by_pairs<T, 8>(a, bwd, interleaved, stream);
  if (lanes <= 16) return by_pairs<T, 16>(a, bwd, interleaved, stream);
  return by_pairs<T, 32>(a, bwd, interleaved, stream);
}

dash_status_t by_type(const Args& a, bool bwd, bool interleaved, int dtype, cudaStream_t stream) {
  if (dtype == DASH_BF16) return by_lanes<__nv_bfloat16>(a, bwd, interleaved, stream);
  if (dtype == DASH_FP16) return by_lanes<__half>(a, bwd, interleaved, stream);
  return by_lanes<float>(a, bwd, interleaved, stream);
}

bool shape_ok(int B, int S, int Hq, int Hk, int D) {
  return B >= 0 && S >= 0 && Hq >= 0 && Hk >= 0 && D >= 8 && D <= kMaxD && D % 8 == 0 && Hq <= (1 << 20) &&
         Hk <= (1 << 20) && (long long)B * S < (1ll << 31) - 256 &&
         (long long)B * S * ((long long)Hq + Hk) < (1ll << 31) - 256;
}

bool strides_ok(const long long* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8 || s[i] < 0 || s[i] > (1ll << 40)) return false;
  return true;
}

// Arguments that both directions share.
dash_status_t check(const void* q, const void* k, const float* wq, const float* wk, const float* cos,
                    const float* sin, const void* positions, int B, int S, int Hq, int Hk, int D, int R,
                    long long P, const long long* qs, const long long* ks, long long pos_stride, float eps,
                    int interleaved, int dtype, int id_bits) {
  if (B < 0 || S < 0 || Hq < 0 || Hk < 0 || D < 1 || R < 0 || R > D || R % 2 || P < 0 || !(eps >= 0.f))
    return DASH_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return DASH_ERR_INVALID_ARG;
  if (dtype != DASH_BF16 && dtype != DASH_FP16 && dtype != DASH_FP32) return DASH_ERR_INVALID_ARG;
  if (id_bits != 32 && id_bits != 64) return DASH_ERR_INVALID_ARG;
  if (!shape_ok(B, S, Hq, Hk, D)) return DASH_ERR_UNSUPPORTED;
  if (!qs || !ks || pos_stride < 0 || pos_stride > (1ll << 40)) return DASH_ERR_INVALID_ARG;
  if (!strides_ok(qs) || !strides_ok(ks)) return DASH_ERR_UNSUPPORTED;
  if ((long long)B * S > 0 && ((Hq > 0 && !q) || (Hk > 0 && !k) || (R > 0 && (!cos || !sin))))
    return DASH_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(wq, 16) || !is_aligned(wk, 16) ||
      !is_aligned(cos, 16) || !is_aligned(sin, 16) || !is_aligned(positions, id_bits / 8))
    return DASH_ERR_INVALID_ARG;
  return DASH_OK;
}

Args common(const void* q, const void* k, const float* wq, const float* wk, const float* cos, const float* sin,
            const void* positions, int B, int S, int Hq, int Hk, int D, int R, long long P, const long long* qs,
            const long long* ks, long long pos_stride, float eps, int id_bits) {
  Args a = {};
  const void* xs[2] = {q, k};
  const float* ws[2] = {wq, wk};
  const long long* st[2] = {qs, ks};
  const int hs[2] = {Hq, Hk};
  for (int i = 0; i < 2; ++i) {
    a.side[i].x = xs[i];
    a.side[i].w = ws[i];
    a.side[i].sb = st[i][0];
    a.side[i].ss = st[i][1];
    a.side[i].sh = st[i][2];
    a.side[i].H = hs[i];
  }
  a.cos = cos;
  a.sin = sin;
  a.pos = positions;
  a.pos_stride = pos_stride;
  // without a rotation no table row is read: every position is in range
  a.P = R > 0 ? P : INT64_MAX;
  a.id_bits = id_bits;
  a.tokens = B * S;
  a.S = S;
  a.D = D;
  a.R = R;
  a.eps = eps;
  return a;
}

}  // namespace

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
  const bool any = (long long)B * S > 0;
  if (any && ((Hq > 0 && !q_out) || (Hk > 0 && !k_out))) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(q_out, 16) || !is_aligned(k_out, 16) || !is_aligned(status, 4)) return DASH_ERR_INVALID_ARG;
  Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride,
                  eps, id_bits);
  void* outs[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    Side& sd = a.side[i];
    sd.out = outs[i];
    sd.oh = D;
    sd.os = (long long)sd.H * D;
    sd.ob = sd.os * S;
  }
  a.status = status;
  if (status) DASH_TRY(cudaMemsetAsync(status, 0, sizeof(int), stream));
  if (!any) return DASH_OK;
  return by_type(a, false, interleaved != 0, dtype, stream);
}

size_t dash_qk_norm_rope_bwd_workspace_size(int B, int S, int Hq, int Hk, int D) {
  if (!shape_ok(B, S, Hq, Hk, D)) return 0;
  return kWsHeaderBytes + round_up_to((size_t)2 * (kBwdBlocks + 1) * (D + 1) * sizeof(float), 256);
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
  if (!workspace || !dq_strides || !dk_strides) return DASH_ERR_INVALID_ARG;
  if (!strides_ok(dq_strides) || !strides_ok(dk_strides)) return DASH_ERR_UNSUPPORTED;
  const bool any = (long long)B * S > 0;
  if (any && ((Hq > 0 && (!dq_out || !dq)) || (Hk > 0 && (!dk_out || !dk)))) return DASH_ERR_INVALID_ARG;
  for (const void* p : {dq_out, dk_out, (const void*)dq, (const void*)dk})
    if (!is_aligned(p, 16)) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(dwq, 4) || !is_aligned(dwk, 4) || !is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  if (workspace_bytes < dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D)) return DASH_ERR_WORKSPACE_TOO_SMALL;
  Args a = common(q, k, wq, wk, cos, sin, positions, B, S, Hq, Hk, D, R, P, q_strides, k_strides, pos_stride,
                  eps, id_bits);
  const void* douts[2] = {dq_out, dk_out};
  void* outs[2] = {dq, dk};
  float* dws[2] = {dwq, dwk};
  const long long* os[2] = {dq_strides, dk_strides};
  float* part = (float*)((char*)workspace + kWsHeaderBytes);
  for (int i = 0; i < 2; ++i) {
    Side& sd = a.side[i];
    sd.dout = douts[i];
    sd.out = outs[i];
    sd.dw = dws[i];
    sd.ob = os[i][0];
    sd.os = os[i][1];
    sd.oh = os[i][2];
    sd.part = part + (size_t)i * (kBwdBlocks + 1) * D;
    sd.bad = (int*)(part + (size_t)2 * (kBwdBlocks + 1) * D) + i * (kBwdBlocks + 1);
  }
  a.header = (int*)workspace;
  return by_type(a, true, interleaved != 0, dtype, stream);
}

}  // extern "C"
