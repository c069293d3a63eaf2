// Norm of queries and keys per head with the rotation in the same pass (dash_qk_norm_rope_*,
// dash_qk_norm_rope_axes_*): the kernels and their launches.
//
// A lane holds two chunks of 8 consecutive values of a head, so a head lies in L = D / 16 lanes
// (rounded up to a power of two) and the mean of squares is a shuffle tree over them. The
// chunks are chosen so that rotation partners meet in one lane: chunks j and j + R / 16 for
// half-split pairs, neighbours for interleaved ones. (Where R / 2 is no multiple of 8, or of 4
// for interleaved pairs, a value's partner is read once more, which hits L1: 16384 tokens x 40
// heads x 96 with R = 24 take 178 us forward and 169 backward, where the bytes take 37 and 56.)
// Both directions read and write every value once: bound by HBM, with the instructions next
// (8 values a lane and shuffled partners took 22 an element forward, 31 backward, and 105 and
// 167 us for 16384 tokens x 64 heads x 128; now 15 and 23, and 232 us for both, where the bytes
// take 200). A warp walks over
// tokens, the grid's warps apart, and copies the next items' rows into its part of
// shared memory while it computes one (cp.async, two items ahead), so that loads are in flight
// all the time without registers; a token's angles are loaded once for all its heads.
// With several axes (AXES) a token has a position for each, and every pair of columns turns by the
// angle of its axis' position: the rows of the angles' tables differ from pair to pair, which only
// the loads of a token's angles see (16 bytes at a time where four pairs share an axis): 252 us for
// both directions of the size above, of it 159 backward, where one axis takes 140. The wait for the
// positions and then the table is what is longer there.
#pragma once

#include <algorithm>

#include "dash_train.h"
#include "host_common.h"
#include "train_common.cuh"

namespace dash {
namespace rope {

using namespace dash::train;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 256;
// Blocks that share the rows: three (forward) and two (backward) for each of 152 SMs, which is
// what an SM holds. The backward's number fixes how dw's sum is split, so it is a constant and
// not the device's SM count.
constexpr int kFwdBlocks = 456;
constexpr int kBwdBlocks = 304;
static_assert(kBwdBlocks + 2 <= 1024, "dw_join looks at all blocks at once");

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
  // A unit of work is one token and gp of its head groups: parts units a token, taken step units
  // apart by a warp. The step in (part, token, batch) digits saves divisions.
  int groups, gp, parts, step_part, step_s, step_b;
  unsigned units, step;
};

struct Args {
  Side side[2];
  const float *cos, *sin;
  const void* pos;
  long long pos_stride, P;
  int id_bits;
  int tokens, S, D, R, interleaved;
  float eps;
  int* header;                      // backward: workspace header
  int* status;                      // forward: optional status word
  // several axes: a position for each, axis_stride elements apart; pair i turns by that of axis
  // (pair_axis[i / 16] >> 2 (i % 16)) & 3
  int axes;
  long long axis_stride;
  uint32_t pair_axis[kMaxD / 32];
};
constexpr int kMaxAxes = 4;

constexpr int kNoToken = 0x7fffffff;

enum Mode : int { HALF = 0, PAIRS = 1, ANY = 2 };

__device__ __forceinline__ void four(const float* p, float* v) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}

// A lane's 16 values: v[0..7] are the columns from c0, v[8..15] those from c1 (at D or beyond:
// not there). Its 8 pairs are (v[i], v[8 + i]) in mode HALF, (v[2i], v[2i + 1]) in mode PAIRS.
template <int M>
struct Lane {
  int c0, c1;
  bool in0, in1;
  __device__ __forceinline__ Lane(const Args& a, int j) {
    // lanes side by side hold chunks side by side, so that a warp's accesses fill whole sectors:
    // the first R / 16 lanes the halves of the rotated columns, the others those of the rest
    const int rot = M == HALF ? a.R >> 4 : 0, from = 16 * rot;
    const int rest = (a.D - from + 15) >> 4;
    c0 = j < rot ? 8 * j : from + 8 * (j - rot);
    c1 = c0 + 8 * (j < rot ? rot : rest);
    if (j >= rot + rest) c0 = c1 = a.D;            // nothing for this lane
    in0 = c0 < a.D;
    in1 = c1 < a.D;
  }
};
template <int M>
__device__ __forceinline__ constexpr int first_of(int i) { return M == HALF ? i : 2 * i; }
template <int M>
__device__ __forceinline__ constexpr int second_of(int i) { return M == HALF ? 8 + i : 2 * i + 1; }

// A token's place: its position, -1 when that is out of range.
template <bool AXES>
struct Place {
  long long p;
  __device__ __forceinline__ Place() : p(0) {}
  __device__ __forceinline__ Place(const Args& a, int b, int s) {
    p = a.pos ? load_index(a.pos, b * a.pos_stride + s, a.id_bits) : (long long)s;
    if (p < 0 || p >= a.P) p = -1;
  }
  __device__ __forceinline__ bool bad() const { return p < 0; }
  // the table row of pair i, and whether pairs i .. i + 3 share it (i a multiple of 4)
  __device__ __forceinline__ long long row(const Args&, int) const { return p; }
  __device__ __forceinline__ bool shared(const Args&, int) const { return true; }
};
// With several axes: a position of each (below 2^31), all of them -1 when one is out of range.
template <>
struct Place<true> {
  int p[kMaxAxes];
  __device__ __forceinline__ Place() : p{} {}
  __device__ __forceinline__ Place(const Args& a, int b, int s) {
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) {
      p[x] = 0;
      if (x < a.axes) {
        const long long v = load_index(a.pos, x * a.axis_stride + b * a.pos_stride + s, a.id_bits);
        bad |= v < 0 || v >= a.P;
        p[x] = (int)v;
      }
    }
    if (bad) p[0] = -1;
  }
  __device__ __forceinline__ bool bad() const { return p[0] < 0; }
  __device__ __forceinline__ uint32_t axes4(const Args& a, int i) const {
    return a.pair_axis[i >> 4] >> (2 * (i & 15));
  }
  __device__ __forceinline__ long long row(const Args& a, int i) const {
    const uint32_t x = axes4(a, i) & 3u;
    return x < 2 ? (x == 0 ? p[0] : p[1]) : (x == 2 ? p[2] : p[3]);
  }
  __device__ __forceinline__ bool shared(const Args& a, int i) const {
    const uint32_t x = axes4(a, i) & 255u;
    return x == 85u * (x & 3u);
  }
};

// cos and sin of the lane's 8 pairs at the token's place (none rotated: a bad place, or columns
// beyond R).
template <int M, bool AXES>
__device__ __forceinline__ void load_angles(const Args& a, const Lane<M>& ln, const Place<AXES>& p, float (&c)[8],
                                            float (&s)[8]) {
  const int half = a.R >> 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {                    // four pairs at a time
    const int col = M == HALF ? ln.c0 + 4 * k : k == 0 ? ln.c0 : ln.c1;
    const bool rotated = !p.bad() && (M == HALF ? ln.c0 < half : col < a.R);
    const int pair = M == HALF ? col : col >> 1;
    if (rotated && p.shared(a, pair)) {
      const long long at = p.row(a, pair) * half + pair;
      four(a.cos + at, c + 4 * k);
      four(a.sin + at, s + 4 * k);
    } else if (rotated) {                          // a border between axes among the four
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = p.row(a, pair + i) * half + pair + i;
        c[4 * k + i] = __ldg(a.cos + at);
        s[4 * k + i] = __ldg(a.sin + at);
      }
    } else {
#pragma unroll
      for (int i = 4 * k; i < 4 * k + 4; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
  }
}

template <int M>
__device__ __forceinline__ void load_weights(const float* w, const Lane<M>& ln, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 1.f;
  if (w && ln.in0) {
    four(w + ln.c0, v);
    four(w + ln.c0 + 4, v + 4);
  }
  if (w && ln.in1) {
    four(w + ln.c1, v + 8);
    four(w + ln.c1 + 4, v + 12);
  }
}

// Mode ANY: rotates the 16 values by themselves (sign +1; -1: the transpose); `partner(c)` gives
// the value of column c.
template <bool AXES, typename F>
__device__ __forceinline__ void rotate_any(const Args& a, const Lane<ANY>& ln, const Place<AXES>& p, bool live,
                                           float sign, float (&y)[16], F partner) {
  const int half = a.R >> 1;
  float z[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = (i < 8 ? ln.c0 : ln.c1) + (i & 7);
    z[i] = y[i];
    if (c < a.R && live && !p.bad()) {
      const bool lo = a.interleaved ? (c & 1) == 0 : c < half;
      const int k = a.interleaved ? c >> 1 : lo ? c : c - half;
      const int o = a.interleaved ? c ^ 1 : lo ? c + half : c - half;
      const long long at = p.row(a, k) * half + k;
      z[i] = y[i] * __ldg(a.cos + at) + (lo ? -sign : sign) * __ldg(a.sin + at) * partner(o);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = z[i];
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp's place in its work: units of one token and `gp` groups of its heads, the grid's warps
// apart (so that together they sweep the tensor in order), group by group.
struct Cursor {
  int b, s, part, grp, end;
  unsigned unit;
  bool fresh;                                     // at the unit's first group
  __device__ __forceinline__ Cursor(const Args& a, const Side& sd, unsigned first) : unit(first) {
    const unsigned token = first / sd.parts;
    part = (int)(first - token * sd.parts);
    b = (int)(token / a.S);
    s = (int)(token - b * a.S);
    start(sd);
  }
  __device__ __forceinline__ bool more(const Side& sd) const { return unit < sd.units; }
  __device__ __forceinline__ void start(const Side& sd) {
    grp = part * sd.gp;
    end = min(grp + sd.gp, sd.groups);
    fresh = true;
  }
  __device__ __forceinline__ void next(const Args& a, const Side& sd) {
    fresh = false;
    if (++grp == end) {                           // step units on, in mixed digits
      unit += sd.step;
      part += sd.step_part;
      s += sd.step_s;
      b += sd.step_b;
      if (part >= sd.parts) {
        part -= sd.parts;
        ++s;
      }
      if (s >= a.S) {
        s -= a.S;
        ++b;
      }
      start(sd);
    }
  }
};

// 8 values from global to shared memory without registers; zeros where `live` is false. A warp's
// 16-byte pieces lie side by side, 512 bytes a piece of every lane. The two pieces of 8 fp32
// values share a sector, which L1 keeps for the second.
template <typename T>
__device__ __forceinline__ void copy8(uint32_t dst, const T* src, bool live) {
  const int n = live ? 16 : 0;
  if constexpr (sizeof(T) == 2) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 512),
                   "l"(reinterpret_cast<const char*>(src) + (live ? i * 16 : 0)), "r"(n)
                   : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ void from_shared(const char* at, float* f) {
  Vec<T, 8> x;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + i * 512);
    x.w[4 * i] = v.x;
    x.w[4 * i + 1] = v.y;
    x.w[4 * i + 2] = v.z;
    x.w[4 * i + 3] = v.w;
  }
  float y[8];
  unpack<T, 8>(x, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = y[i];
}
// 8 fp32 values in one store where the address allows it: a whole sector.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if (sizeof(T) == 4 && ((uintptr_t)p & 31) == 0)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  else
    store_f32<T, 8>(p, x);
}
template <typename T, int M>
__device__ __forceinline__ void store16(T* row, const Lane<M>& ln, const float (&v)[16]) {
  float x[8];
  if (ln.in0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
    store8<T>(row + ln.c0, x);
  }
  if (ln.in1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[8 + i];
    store8<T>(row + ln.c1, x);
  }
}

// Items in shared memory beside the one in work: two of U groups of heads. The backward takes
// one group an item, which needs fewer registers, and as many bytes ahead.
template <typename T, bool BWD>
constexpr int kItemsAhead = BWD && sizeof(T) == 2 ? 4 : 2;

// Bytes of one row of every lane group of a warp: 8 values a lane, twice.
template <typename T>
constexpr int kChunkBytes = 32 * 8 * (int)sizeof(T);
template <typename T, int U, bool BWD>
constexpr int kSharedBytes = kWarps * (kItemsAhead<T, BWD> + 1) * U * (BWD ? 4 : 2) * kChunkBytes<T>;

template <typename T, int L, int M, int U, bool AXES>
__global__ void __launch_bounds__(kThreads, M == ANY ? 2 : 3) fwd_kernel(const Args a) {
  constexpr int RW = 32 / L, kAhead = kItemsAhead<T, false>, kStages = kAhead + 1;   // RW: heads a warp handles at once
  extern __shared__ char qk_smem[];
  const int which = blockIdx.x >= a.side[0].blocks;
  const Side& sd = a.side[which];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L;
  const Lane<M> ln(a, lane % L);
  const float inv_d = 1.f / a.D;
  char* mine = qk_smem + warp * (kStages * U * 2 * kChunkBytes<T>) + lane * 16;
  const uint32_t mine_s = (uint32_t)__cvta_generic_to_shared(mine);
  Cursor at(a, sd, (blockIdx.x - (which ? a.side[0].blocks : 0)) * kWarps + warp);
  Cursor ahead = at;
  auto fetch = [&](int stage) {                    // the item at `ahead`; an empty group past the end
    if (ahead.more(sd)) {
      const T* x = (const T*)sd.x + ahead.b * sd.sb + ahead.s * sd.ss;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (ahead.grp * U + u) * RW + sub;
        const bool live = h < sd.H;
        const T* row = live ? x + h * sd.sh : (const T*)sd.x;
        const uint32_t to = mine_s + (stage * U + u) * 2 * kChunkBytes<T>;
        copy8<T>(to, live && ln.in0 ? row + ln.c0 : row, live && ln.in0);
        copy8<T>(to + kChunkBytes<T>, live && ln.in1 ? row + ln.c1 : row, live && ln.in1);
      }
      ahead.next(a, sd);
    }
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(k);
  // a pair's output is r (x_a (w_a c) - x_b (w_b s)), r (x_b (w_b c) + x_a (w_a s))
  float ac[8], bs[8], bc[8], as[8], w[16];
  if (M == ANY) load_weights(sd.w, ln, w);
  Place<AXES> p;
  for (int stage = 0; at.more(sd);) {
    fetch(stage >= 1 ? stage - 1 : kStages - 1);   // into the stage that the last item left
    if (at.fresh) {
      p = Place<AXES>(a, at.b, at.s);
      if (p.bad() && a.status) *a.status = kStatusBounds;
      if constexpr (M != ANY) {
        float c[8], s[8];
        load_weights(sd.w, ln, w);
        load_angles<M, AXES>(a, ln, p, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wa = w[first_of<M>(i)], wb = w[second_of<M>(i)];
          ac[i] = wa * c[i];
          bs[i] = wb * s[i];
          bc[i] = wb * c[i];
          as[i] = wa * s[i];
        }
      }
    }
    copies_wait<kAhead>();
    T* out = (T*)sd.out + at.b * sd.ob + at.s * sd.os;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (at.grp * U + u) * RW + sub;
      float x[16], q0 = 0.f, q1 = 0.f;
      const char* from = mine + (stage * U + u) * 2 * kChunkBytes<T>;
      from_shared<T>(from, x);
      from_shared<T>(from + kChunkBytes<T>, x + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        q0 = fmaf(x[i], x[i], q0);
        q1 = fmaf(x[8 + i], x[8 + i], q1);
      }
      const float r = p.bad() ? NAN : rsqrtf(lanes_sum<L>(q0 + q1) * inv_d + a.eps);
      float y[16];
      if constexpr (M == ANY) {
        const T* row = (const T*)sd.x + at.b * sd.sb + at.s * sd.ss + h * sd.sh;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = x[i] * w[i] * r;
        rotate_any<AXES>(a, ln, p, h < sd.H, 1.f, y, [&](int c) {
          return to_f32(row[c]) * (sd.w ? __ldg(sd.w + c) : 1.f) * r;
        });
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xa = x[first_of<M>(i)], xb = x[second_of<M>(i)];
          y[first_of<M>(i)] = (xa * ac[i] - xb * bs[i]) * r;
          y[second_of<M>(i)] = (xb * bc[i] + xa * as[i]) * r;
        }
      }
      if (h < sd.H) store16<T, M>(out + h * sd.oh, ln, y);
    }
    at.next(a, sd);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
}

// Backward: the same walk over the rows of x and of the output's gradient. With e the rotated
// gradient, t = e x and m = sum(w t) / D: dw += r t, dx = r (w e - r^2 m x). A warp keeps its
// columns' part of dw in registers; the block's warps are added in order.
template <typename T, int L, int M, int U, bool AXES>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(const Args a) {
  constexpr int RW = 32 / L, kAhead = kItemsAhead<T, true>, kStages = kAhead + 1;
  extern __shared__ char qk_smem[];
  __shared__ float dws[kWarps][kMaxD];
  __shared__ int bad;
  grid_next();
  if (threadIdx.x == 0) bad = kNoToken;
  __syncthreads();
  const int which = blockIdx.x >= a.side[0].blocks;
  const Side& sd = a.side[which];
  const int block = blockIdx.x - (which ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L;
  const Lane<M> ln(a, lane % L);
  const float inv_d = 1.f / a.D;
  char* mine = qk_smem + warp * (kStages * U * 4 * kChunkBytes<T>) + lane * 16;
  const uint32_t mine_s = (uint32_t)__cvta_generic_to_shared(mine);
  Cursor at(a, sd, (unsigned)block * kWarps + warp);
  Cursor ahead = at;
  auto fetch = [&](int stage) {
    if (ahead.more(sd)) {
      const T* x = (const T*)sd.x + ahead.b * sd.sb + ahead.s * sd.ss;
      const T* d = (const T*)sd.dout + ((long long)ahead.b * a.S + ahead.s) * sd.H * a.D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (ahead.grp * U + u) * RW + sub;
        const bool live = h < sd.H, l0 = live && ln.in0, l1 = live && ln.in1;
        const T* xr = live ? x + h * sd.sh : (const T*)sd.x;
        const T* dr = live ? d + h * a.D : (const T*)sd.dout;
        const uint32_t to = mine_s + (stage * U + u) * 4 * kChunkBytes<T>;
        copy8<T>(to, l0 ? xr + ln.c0 : xr, l0);
        copy8<T>(to + kChunkBytes<T>, l1 ? xr + ln.c1 : xr, l1);
        copy8<T>(to + 2 * kChunkBytes<T>, l0 ? dr + ln.c0 : dr, l0);
        copy8<T>(to + 3 * kChunkBytes<T>, l1 ? dr + ln.c1 : dr, l1);
      }
      ahead.next(a, sd);
    }
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(k);
  float w[16], dw[16] = {}, c[8], s[8];
  load_weights(sd.w, ln, w);
  Place<AXES> p;
  for (int stage = 0; at.more(sd);) {
    fetch(stage >= 1 ? stage - 1 : kStages - 1);
    if (at.fresh) {
      p = Place<AXES>(a, at.b, at.s);
      if (p.bad() && lane == 0) atomicMin(&bad, at.b * a.S + at.s);
      if constexpr (M != ANY) load_angles<M, AXES>(a, ln, p, c, s);
    }
    copies_wait<kAhead>();
    T* out = (T*)sd.out + at.b * sd.ob + at.s * sd.os;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (at.grp * U + u) * RW + sub;
      float x[16], e[16], q0 = 0.f, q1 = 0.f;
      const char* from = mine + (stage * U + u) * 4 * kChunkBytes<T>;
      from_shared<T>(from, x);
      from_shared<T>(from + kChunkBytes<T>, x + 8);
      from_shared<T>(from + 2 * kChunkBytes<T>, e);
      from_shared<T>(from + 3 * kChunkBytes<T>, e + 8);
      if constexpr (M == ANY) {
        const T* row = (const T*)sd.dout + (((long long)at.b * a.S + at.s) * sd.H + h) * a.D;
        rotate_any<AXES>(a, ln, p, h < sd.H, -1.f, e, [&](int col) { return to_f32(row[col]); });
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float da = e[first_of<M>(i)], db = e[second_of<M>(i)];
          e[first_of<M>(i)] = da * c[i] + db * s[i];
          e[second_of<M>(i)] = db * c[i] - da * s[i];
        }
      }
      float m0 = 0.f, m1 = 0.f, t[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        q0 = fmaf(x[i], x[i], q0);
        q1 = fmaf(x[8 + i], x[8 + i], q1);
        t[i] = e[i] * x[i];
        t[8 + i] = e[8 + i] * x[8 + i];
        m0 = fmaf(w[i], t[i], m0);
        m1 = fmaf(w[8 + i], t[8 + i], m1);
      }
      const float r = p.bad() ? NAN : rsqrtf(lanes_sum<L>(q0 + q1) * inv_d + a.eps);
      const float k = r * r * (lanes_sum<L>(m0 + m1) * inv_d);
      const float rd = h < sd.H ? r : 0.f;         // rows that are not there are all zeros
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        dw[i] = fmaf(rd, t[i], dw[i]);
        e[i] = fmaf(-k, x[i], e[i] * w[i]) * r;
      }
      if (h < sd.H) store16<T, M>(out + h * sd.oh, ln, e);
    }
    at.next(a, sd);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  // heads of the warp, then warps, in order
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
    if (sub == 0 && (i < 8 ? ln.in0 : ln.in1)) dws[warp][(i < 8 ? ln.c0 : ln.c1) + (i & 7)] = dw[i];
  }
  __syncthreads();
  for (int col = threadIdx.x; col < a.D; col += kThreads) {
    float t = 0.f;
    for (int k = 0; k < kWarps; ++k) t += dws[k][col];
    sd.part[(long long)block * a.D + col] = t;
  }
  if (threadIdx.x == 0) sd.bad[block] = bad;
}

// dw = the blocks' parts, added in order: 32 groups of consecutive blocks, then the groups.
// One block for each 32 columns of one tensor; the first also writes the call's status.
template <bool AXES>
__global__ void __launch_bounds__(1024) dw_join_kernel(const Args a) {
  __shared__ float sums[32][33];
  __shared__ int first;
  grid_wait();
  const Side& sd = a.side[blockIdx.x];
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) first = kNoToken;
    __syncthreads();
    const int n = a.side[0].blocks, b = threadIdx.x;      // at most kBwdBlocks + 2
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
        if (threadIdx.x == WS_EXPECT && a.pos)
          for (int x = 0; x < (AXES ? a.axes : 1); ++x) {      // the first axis that is out of range
            const long long q = load_index(a.pos, x * a.axis_stride + first / a.S * a.pos_stride + first % a.S, a.id_bits);
            v = (int)q;
            if (q < 0 || q >= a.P) break;
          }
        if (threadIdx.x == WS_EXPECT && !a.pos) v = first % a.S;
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

template <typename T, int L, int M, bool AXES>
dash_status_t launch(Args a, bool bwd, cudaStream_t stream) {
  constexpr int RW = 32 / L;
  constexpr int UF = sizeof(T) == 4 ? 1 : 2;
  // heads in flight a warp: U when that leaves every warp of the chip (about 10^4) an item,
  // else one, which spreads few tokens over more warps
  const long long rows = (long long)a.tokens * (a.side[0].H + a.side[1].H);
  const bool many = !bwd && rows / (UF * RW) >= 9728;
  const int per = many ? UF * RW : RW;
  // each tensor's share of the blocks goes by its heads
  const int H = a.side[0].H + a.side[1].H, most = bwd ? kBwdBlocks : kFwdBlocks;
  for (int i = 0; i < 2; ++i) {
    const long long items = (long long)a.tokens * ceil_div(a.side[i].H, per);
    const long long share = H > 0 ? std::max<long long>(1, ((long long)most * a.side[i].H + H / 2) / H) : 0;
    a.side[i].blocks = (int)std::min<long long>(ceil_div<long long>(items, kWarps), share);
    // whole tokens a unit when every warp gets several, else parts of them
    Side& sd = a.side[i];
    const long long warps = (long long)sd.blocks * kWarps;
    sd.groups = std::max(1, ceil_div(sd.H, per));
    const long long parts = a.tokens > 0 ? std::min<long long>(sd.groups, ceil_div<long long>(4 * warps, a.tokens)) : 1;
    sd.gp = (int)ceil_div<long long>(sd.groups, std::max<long long>(parts, 1));
    sd.parts = ceil_div(sd.groups, sd.gp);
    sd.units = (unsigned)a.tokens * sd.parts;
    sd.step = (unsigned)warps;
    sd.step_part = (int)(warps % sd.parts);
    const long long tokens = warps / sd.parts;
    sd.step_s = a.S > 0 ? (int)(tokens % a.S) : 0;
    sd.step_b = a.S > 0 ? (int)(tokens / a.S) : 0;
  }
  const unsigned grid = a.side[0].blocks + a.side[1].blocks;
  if (grid > 0) {
    const auto kernel = bwd ? bwd_kernel<T, L, M, 1, AXES>
                            : many ? fwd_kernel<T, L, M, UF, AXES> : fwd_kernel<T, L, M, 1, AXES>;
    const int smem = bwd ? kSharedBytes<T, 1, true> : many ? kSharedBytes<T, UF, false> : kSharedBytes<T, 1, false>;
    DASH_TRY(allow_shared((const void*)kernel, smem));
    kernel<<<grid, kThreads, smem, stream>>>(a);
    DASH_TRY(cudaGetLastError());
  }
  if (bwd) DASH_TRY(launch_after(dw_join_kernel<AXES>, dim3(2, ceil_div(a.D, 32)), 1024, 0, stream, a));
  return DASH_OK;
}

template <typename T, int L, bool AXES>
dash_status_t by_pairs(const Args& a, bool bwd, cudaStream_t stream) {
  if (a.interleaved && a.R % 8 == 0) return launch<T, L, PAIRS, AXES>(a, bwd, stream);
  if (!a.interleaved && a.R % 16 == 0) return launch<T, L, HALF, AXES>(a, bwd, stream);
  return launch<T, L, ANY, AXES>(a, bwd, stream);
}

template <typename T, bool AXES>
dash_status_t by_lanes(const Args& a, bool bwd, cudaStream_t stream) {
  if (a.D <= 64) return by_pairs<T, 4, AXES>(a, bwd, stream);
  if (a.D <= 128) return by_pairs<T, 8, AXES>(a, bwd, stream);
  return by_pairs<T, 16, AXES>(a, bwd, stream);
}

template <bool AXES>
dash_status_t by_type(const Args& a, bool bwd, int dtype, cudaStream_t stream) {
  if (dtype == DASH_BF16) return by_lanes<__nv_bfloat16, AXES>(a, bwd, stream);
  if (dtype == DASH_FP16) return by_lanes<__half, AXES>(a, bwd, stream);
  return by_lanes<float, AXES>(a, bwd, stream);
}

// Arguments that both directions and both operators share.
inline bool shape_ok(int B, int S, int Hq, int Hk, int D) {
  return B >= 0 && S >= 0 && Hq >= 0 && Hk >= 0 && D >= 8 && D <= kMaxD && D % 8 == 0 && Hq <= (1 << 20) &&
         Hk <= (1 << 20) && (long long)B * S < (1ll << 31) - 256 &&
         (long long)B * S * ((long long)Hq + Hk) < (1ll << 31) - 256;
}

inline bool strides_ok(const long long* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8 || s[i] < 0 || s[i] > (1ll << 40)) return false;
  return true;
}

// Strides of a tensor to write: no two of its elements in one place by a stride of zero.
inline bool distinct(const long long* s, int B, int S, int H) {
  return (B < 2 || s[0] > 0) && (S < 2 || s[1] > 0) && (H < 2 || s[2] > 0);
}

inline dash_status_t check(const void* q, const void* k, const float* wq, const float* wk, const float* cos,
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

inline Args common(const void* q, const void* k, const float* wq, const float* wk, const float* cos, const float* sin,
            const void* positions, int B, int S, int Hq, int Hk, int D, int R, long long P, const long long* qs,
            const long long* ks, long long pos_stride, float eps, int interleaved, int id_bits) {
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
  a.interleaved = interleaved;
  return a;
}

template <bool AXES>
dash_status_t run_fwd(Args a, void* q_out, void* k_out, int* status, int dtype, cudaStream_t stream) {
  if (a.tokens > 0 && ((a.side[0].H > 0 && !q_out) || (a.side[1].H > 0 && !k_out))) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(q_out, 16) || !is_aligned(k_out, 16) || !is_aligned(status, 4)) return DASH_ERR_INVALID_ARG;
  void* outs[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    Side& sd = a.side[i];
    sd.out = outs[i];
    sd.oh = a.D;
    sd.os = (long long)sd.H * a.D;
    sd.ob = sd.os * a.S;
  }
  a.status = status;
  if (status) DASH_TRY(cudaMemsetAsync(status, 0, sizeof(int), stream));
  if (a.tokens == 0) return DASH_OK;
  return by_type<AXES>(a, false, dtype, stream);
}

inline size_t bwd_workspace_size(int B, int S, int Hq, int Hk, int D) {
  if (!shape_ok(B, S, Hq, Hk, D)) return 0;
  return kWsHeaderBytes + round_up_to((size_t)2 * (kBwdBlocks + 1) * (D + 1) * sizeof(float), 256);
}

template <bool AXES>
dash_status_t run_bwd(Args a, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                      void* workspace, size_t workspace_bytes, int B, const long long* dq_strides,
                      const long long* dk_strides, int dtype, cudaStream_t stream) {
  const int S = a.S, Hq = a.side[0].H, Hk = a.side[1].H, D = a.D;
  if (!workspace || !dq_strides || !dk_strides) return DASH_ERR_INVALID_ARG;
  if (!strides_ok(dq_strides) || !strides_ok(dk_strides)) return DASH_ERR_UNSUPPORTED;
  if (!distinct(dq_strides, B, S, Hq) || !distinct(dk_strides, B, S, Hk)) return DASH_ERR_INVALID_ARG;
  if (a.tokens > 0 && ((Hq > 0 && (!dq_out || !dq)) || (Hk > 0 && (!dk_out || !dk)))) return DASH_ERR_INVALID_ARG;
  for (const void* p : {dq_out, dk_out, (const void*)dq, (const void*)dk})
    if (!is_aligned(p, 16)) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(dwq, 4) || !is_aligned(dwk, 4) || !is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  if (workspace_bytes < bwd_workspace_size(B, S, Hq, Hk, D)) return DASH_ERR_WORKSPACE_TOO_SMALL;
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
  return by_type<AXES>(a, true, dtype, stream);
}

}  // namespace rope
}  // namespace dash
