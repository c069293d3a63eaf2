// Group norm with an activation over channels-last tensors and its gradient (dash_group_norm_*).
//
// x [N, S, C], channels c of group g = c / (C / G): xh = (x - mean) rstd, z = xh w + b, y = act(z).
// All sums are sums over rows per channel, in a fixed order: forward s = sum(x - K), q = sum((x -
// K)^2) with the channel's pivot K, the median of five of its values at rows spread over the sample;
// backward A = sum dz, B = rstd sum dz (x - mean) with dz = dy act'(z). Of these come, per group,
//   mean, var            from m_c = K + s / S and q - s^2 / S, joined over the group's channels
//   c1 = mean(w A), c2 = mean(w B);  dx = rstd (w dz - c1 - xh c2),  dw = sum_n B, db = sum_n A.
//
// Two ways, by whether a sample's slab of whole groups fits the shared memory of a cluster:
//  - resident: a cluster takes a slab of channels of one sample, each CTA a range of rows, which it
//    keeps in shared memory (a thread its own 16-byte pieces): x (backward: x and dy) is read once
//    and the call is one kernel. The channel sums meet through distributed shared memory.
//  - in passes: blocks of rows sum into a workspace, a small kernel joins, blocks of rows apply. x is
//    read twice, the second time from L2 as far as it is still there: the second pass runs
//    backwards through the tensor.
// Large maps are bound by memory, the backward's activation by instructions next (of its kernels of 8
// channels a thread the sums and the resident one spill 40 bytes at 64 registers, apply 32): 2 x 65536 x 512
// bf16 (in passes) takes 68 us forward, where 403 MB take 60, and 119 backward, where 671 MB take 99 (sums
// 50 for 40, apply 62 for 59); 4 x 4096 x 512 takes 14 (resident) and 29 (in passes).
#include <algorithm>
#include <climits>

#include "dash_train.h"
#include "host_common.h"
#include "tc_ptx.cuh"
#include "train_common.cuh"

namespace {

using namespace dash;
using namespace dash::train;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Work is cut for a chip of 152 SMs whatever the device has.
constexpr int kChip = 152;
constexpr int kMaxShared = 232448;   // a CTA's shared memory at most

enum Act : int { NONE = 0, SILU = 1 };

struct Args {
  const void* x;
  const void* dy;
  void* out;                 // y or dx, contiguous
  const float *w, *b;
  float *mean, *rstd;        // [N, G]
  float *dw, *db;
  float2* part;              // passes: [N][chunk][C]; sums over a chunk of rows
  float2* chan;              // backward: [N][C] (A, B)
  float2* coef;              // passes, backward: [N][G] (c1, c2)
  long long sb, ss;          // strides of x
  int N, S, C, G, cpg;
  float eps;
  int slab, slabs;           // channels of a slab, slabs of a sample
  int rows;                  // resident: rows of a CTA; passes: rows of a chunk
  int chunks;
  int cols;                  // passes: pieces of a row a block takes
};

// A thread's V consecutive channels.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// 1 / (1 + exp(-z)); the reciprocal of infinity is 0. Within (7 + |z|) 2^-24 of itself, also for fp32 tensors:
// with expf and a reciprocal rounded to nearest an fp32 y is 8.7e-8 off in norm, with these 8.9e-8, and the calls
// take 7 to 14 % longer (bf16: 30 to 45).
__device__ __forceinline__ float sigmoid(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-z)));
  return r;
}
template <int ACT>
__device__ __forceinline__ float activate(float z) { return ACT == SILU ? z * sigmoid(z) : z; }
// dy times the activation's derivative at z
template <int ACT>
__device__ __forceinline__ float activate_grad(float dy, float z) {
  if (ACT == NONE) return dy;
  const float s = sigmoid(z);
  return dy * fmaf(s, fmaf(-z, s, z), s);          // s + s z (1 - s)
}

template <int V>
__device__ __forceinline__ void load_channels(const float* p, int c, float other, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = p ? __ldg(p + c + i) : other;
}

// The pivots of V channels of a sample (x: its first row's; S > 0). Sums around a pivot lose what
// (K - mean)^2 exceeds the variance by, so one value is not enough: with the first row of a map (a
// corner, which padding makes unlike the rest) 300 spreads away, 65536 rows lost 1e-3 of the variance. A
// median of five rows is as far off only where three of the five are, and such rows are much of the spread.
__device__ __forceinline__ float median(float a, float b, float c, float d, float e) {
  const float lo = fmaxf(fminf(a, b), fminf(c, d)), hi = fminf(fmaxf(a, b), fmaxf(c, d));
  return fmaxf(fminf(lo, hi), fminf(fmaxf(lo, hi), e));
}
template <typename T, int V>
__device__ __forceinline__ void load_pivots(const T* x, long long ss, int S, float (&m)[V]) {
  Vec<T, V> row[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) row[k] = load_vec<T, V>(x + (long long)S * (2 * k + 1) / 10 * ss);
  float f[5][V];
#pragma unroll
  for (int k = 0; k < 5; ++k) unpack<T, V>(row[k], f[k]);
#pragma unroll
  for (int i = 0; i < V; ++i) m[i] = median(f[0][i], f[1][i], f[2][i], f[3][i], f[4][i]);
}

// Adds V values to their channels' sums. Forward: m the pivots; backward: z = (x - m) w + b, with
// w holding w rstd. With the activation two channels at a time, as the instructions are what its
// sums take longest; the sums' signs are then turned (kTurned), which saves turning each value's
// (8 x 4096 x 320 bf16: 29.6 us, now 27.5; 4 x 16384 x 128 fp32: 25.6, now 23.9).
template <int V, int ACT, bool BWD>
constexpr bool kTurned = BWD && ACT == SILU && V % 2 == 0;
template <int V, int ACT, bool BWD>
__device__ __forceinline__ void add_sums(const float (&f)[V], const float (&d)[V], const float (&m)[V],
                                         const float (&w)[V], const float (&b)[V], float (&s)[V], float (&q)[V]) {
  if constexpr (kTurned<V, ACT, BWD>) {
    const uint64_t one = two(-1.f, -1.f), log2e = two(-1.4426950408889634f, -1.4426950408889634f);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint64_t t = add2(two(f[i], f[i + 1]), two(-m[i], -m[i + 1]));
      const uint64_t z = fma2(t, two(w[i], w[i + 1]), two(b[i], b[i + 1]));
      float e0, e1, p0, p1;
      untwo(mul2(z, log2e), e0, e1);
      untwo(fma2(two(ptx::ex2(e0), ptx::ex2(e1)), one, one), e0, e1);   // -1 - exp(-z)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(e0));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(e1));
      const uint64_t ns = two(p0, p1);             // minus the sigmoid
      const uint64_t u = mul2(two(d[i], d[i + 1]), fma2(ns, fma2(z, ns, z), ns));
      untwo(add2(two(s[i], s[i + 1]), u), s[i], s[i + 1]);
      untwo(fma2(u, t, two(q[i], q[i + 1])), q[i], q[i + 1]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = f[i] - m[i];
    const float u = BWD ? activate_grad<ACT>(d[i], fmaf(t, w[i], b[i])) : t;
    s[i] += u;
    q[i] = fmaf(u, t, q[i]);
  }
}

template <int V, int ACT, bool BWD>
__device__ __forceinline__ void turn_back(float (&s)[V], float (&q)[V]) {
  if constexpr (kTurned<V, ACT, BWD>) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = -s[i];
      q[i] = -q[i];
    }
  }
}

// With t = x - mean: y = act(t a + b), dx = dz a + t k2 + k1 with a = w rstd, k2 = -rstd^2 c2, k1 = -rstd c1.
// (The mean's part taken into b and k1 would save the subtraction and leave an error of 2^-24 |mean| rstd w: 0.02
// in a group of one value, 1000, whose rstd is 1 / sqrt(eps).)
template <int V, int ACT, bool BWD>
__device__ __forceinline__ void apply(float (&f)[V], const float (&d)[V], const float (&m)[V], const float (&a)[V],
                                      const float (&b)[V], const float (&k1)[V], const float (&k2)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = f[i] - m[i], z = fmaf(t, a[i], b[i]);
    if (BWD) f[i] = fmaf(activate_grad<ACT>(d[i], z), a[i], fmaf(t, k2[i], k1[i]));
    else f[i] = activate<ACT>(z);
  }
}

// Row lanes' sums in block_sums: a warp's lanes are added first where pieces of a row are few.
__host__ __device__ constexpr bool by_warps(int nv) { return nv <= 16 && (nv & (nv - 1)) == 0; }
__host__ __device__ constexpr int sum_rows(int nv) { return by_warps(nv) ? kWarps : kThreads / nv; }

// Sums of a block's threads that hold the same channels: thread t holds channels V (t % nv) of row
// lane t / nv. `red` has room for sum_rows(nv) * nv * V entries; channel c's sum goes to out[c].
template <int V>
__device__ __forceinline__ void block_sums(float (&s)[V], float (&q)[V], int nv, float2* red, float2* out) {
  const int t = threadIdx.x, cs = nv * V;
  int lanes = kThreads / nv;                       // row lanes; the threads beyond them hold zeros
  int row = t / nv;
  const int v = t - row * nv;
  bool mine = row < lanes;
  if (by_warps(nv)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= nv) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
          q[i] += __shfl_xor_sync(0xffffffffu, q[i], o);
        }
      }
    }
    lanes = kWarps;
    row = t >> 5;
    mine = (t & 31) < nv;
  }
  if (mine) {
#pragma unroll
    for (int i = 0; i < V; ++i) red[row * cs + v * V + i] = make_float2(s[i], q[i]);
  }
  __syncthreads();
  // parts of the row lanes, then the parts
  const int parts = max(1, min(kThreads / cs, lanes));
  if (parts > 1) {
    const int part = t / cs, c = t - part * cs;
    float2 a = make_float2(0.f, 0.f);
    if (part < parts)
      for (int r = part; r < lanes; r += parts) {
        const float2 x = red[r * cs + c];
        a.x += x.x;
        a.y += x.y;
      }
    __syncthreads();
    if (part < parts) red[part * cs + c] = a;
    __syncthreads();
    lanes = parts;
  }
  for (int c = t; c < cs; c += kThreads) {
    float2 a = make_float2(0.f, 0.f);
    for (int r = 0; r < lanes; ++r) {
      const float2 x = red[r * cs + c];
      a.x += x.x;
      a.y += x.y;
    }
    out[c] = a;
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Mean and 1 / sqrt(var + eps) of a group (one warp) from its channels' pivots and sums: with m_c
// their means, relative to the first channel's pivot, the squares are those within the channels
// and S times those of the m_c around their mean.
template <typename P, typename F>
__device__ __forceinline__ void group_stats(const Args& a, P pivot, F sums, float* mean, float* rstd) {
  const int lane = threadIdx.x & 31;
  const float n = (float)a.S, k0 = pivot(0);
  float d1 = 0.f, in = 0.f;
  for (int c = lane; c < a.cpg; c += 32) {
    const float2 x = sums(c);
    const float m = x.x / n;
    d1 += pivot(c) - k0 + m;
    in += fmaxf(0.f, x.y - x.x * m);
  }
  const float dm = warp_sum(d1) / a.cpg;
  float d2 = 0.f;
  for (int c = lane; c < a.cpg; c += 32) {
    const float d = pivot(c) - k0 + sums(c).x / n - dm;
    d2 = fmaf(d, d, d2);
  }
  const float var = (warp_sum(in) / n + warp_sum(d2)) / a.cpg;
  *mean = a.S > 0 ? k0 + dm : 0.f;
  *rstd = rsqrtf((a.S > 0 ? var : 0.f) + a.eps);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float2 peer_load(const float2* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(ptx::peer_smem(p, rank)) : "memory");
  return v;
}

// One piece of V channels to this thread's place in shared memory (own: read back by itself).
template <typename T, int V>
__device__ __forceinline__ void fetch_piece(char* to, const T* from) {
  if constexpr (V > 1) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
  } else {
    *reinterpret_cast<T*>(to) = *from;
  }
}
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <typename T, int V>
__device__ __forceinline__ void read_piece(const char* at, float (&f)[V]) {
  if constexpr (V > 1) {
    load_f32<T, V>(reinterpret_cast<const T*>(at), f);
  } else {
    f[0] = to_f32(*reinterpret_cast<const T*>(at));
  }
}
template <typename T, int V>
__device__ __forceinline__ void write_piece(T* to, const float (&f)[V]) {
  if constexpr (V > 1) store_f32<T, V>(to, f);
  else *to = from_f32<T>(f[0]);
}

// Where a resident CTA's thread is: its slab's channels, its rows.
template <int V>
struct Seat {
  int n, c0, cs, nv, v, row, lanes, r0, r1;
  bool on;
  __device__ __forceinline__ Seat(const Args& a, int cluster, int rank) {
    n = cluster / a.slabs;
    c0 = (cluster - n * a.slabs) * a.slab;
    cs = min(a.slab, a.C - c0);
    nv = cs / V;
    lanes = kThreads / nv;
    row = (int)threadIdx.x / nv;
    v = (int)threadIdx.x - row * nv;
    on = row < lanes;
    r0 = rank * a.rows;
    r1 = min(a.S, r0 + a.rows);
  }
};

// Resident, both directions. Shared memory: the pieces (x, then dy), the sums.
template <typename T, int V, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) resident_kernel(const __grid_constant__ Args a, int pieces) {
  constexpr int PB = V * (int)sizeof(T);
  extern __shared__ __align__(16) char gn_smem[];
  char* xs = gn_smem + threadIdx.x * PB;
  char* ds = xs + (size_t)pieces * kThreads * PB;
  float2* sums = (float2*)(gn_smem + (((BWD ? 2 : 1) * pieces * kThreads * PB + 15) & ~15));   // [slab] this CTA's
  float2* total = sums + a.slab;                   // [slab] the cluster's
  float2* grp = total + a.slab;                    // [groups] mean, rstd; backward: c1, c2
  float* pivots = (float*)(grp + a.slab / a.cpg);  // [slab] forward
  float2* red = grp + a.slab / a.cpg + (BWD ? 0 : (a.slab + 1) / 2);
  if (BWD) grid_next();
  const int ranks = (int)cluster_size(), rank = (int)ptx::cluster_rank();
  const Seat<V> st(a, blockIdx.x / ranks, rank);
  const int c = st.c0 + st.v * V, g0 = st.c0 / a.cpg, groups = st.cs / a.cpg;
  const T* x = (const T*)a.x + st.n * a.sb;
  const long long cont = (long long)st.n * a.S * a.C;
  const T* dy = (const T*)a.dy + cont;
  T* out = (T*)a.out + cont;
  if (st.on) {
    int k = 0;
    for (int r = st.r0 + st.row; r < st.r1; r += st.lanes, ++k) {
      fetch_piece<T, V>(xs + (size_t)k * kThreads * PB, x + r * a.ss + c);
      if (BWD) fetch_piece<T, V>(ds + (size_t)k * kThreads * PB, dy + (long long)r * a.C + c);
    }
  }
  float w[V], b[V], m[V], s[V] = {}, q[V] = {};
  if (st.on) {
    load_channels<V>(a.w, c, 1.f, w);
    load_channels<V>(a.b, c, 0.f, b);
    if constexpr (BWD) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = st.n * a.G + (c + i) / a.cpg;
        m[i] = __ldg(a.mean + g);
        w[i] *= __ldg(a.rstd + g);
      }
    } else {
      load_pivots<T, V>(x + c, a.ss, a.S, m);
      if (st.row == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) pivots[st.v * V + i] = m[i];
      }
    }
  }
  fetch_wait();
  if (st.on) {
    int k = 0;
    for (int r = st.r0 + st.row; r < st.r1; r += st.lanes, ++k) {
      float f[V], d[V];
      read_piece<T, V>(xs + (size_t)k * kThreads * PB, f);
      if constexpr (BWD) read_piece<T, V>(ds + (size_t)k * kThreads * PB, d);
      add_sums<V, ACT, BWD>(f, d, m, w, b, s, q);
    }
  }
  turn_back<V, ACT, BWD>(s, q);
  block_sums<V>(s, q, st.nv, red, sums);
  cluster_arrive();
  cluster_wait();
  for (int e = threadIdx.x; e < st.cs; e += kThreads) {
    float2 t = make_float2(0.f, 0.f);
    for (int k = 0; k < ranks; ++k) {
      const float2 y = peer_load(sums + e, k);
      t.x += y.x;
      t.y += y.y;
    }
    if (BWD) t.y *= __ldg(a.rstd + st.n * a.G + (st.c0 + e) / a.cpg);
    total[e] = t;
    if (BWD && rank == 0) a.chan[(long long)st.n * a.C + st.c0 + e] = t;
  }
  cluster_arrive();                                // the peers' sums have been read here
  __syncthreads();
  for (int g = threadIdx.x >> 5; g < groups; g += kWarps) {
    const int lane = threadIdx.x & 31, ch = g * a.cpg;
    if constexpr (BWD) {
      float c1 = 0.f, c2 = 0.f;
      for (int e = lane; e < a.cpg; e += 32) {
        const float wc = a.w ? __ldg(a.w + st.c0 + ch + e) : 1.f;
        c1 = fmaf(wc, total[ch + e].x, c1);
        c2 = fmaf(wc, total[ch + e].y, c2);
      }
      const float n = (float)a.S * (float)a.cpg;
      c1 = warp_sum(c1) / n;
      c2 = warp_sum(c2) / n;
      if (lane == 0) grp[g] = make_float2(c1, c2);
    } else {
      float mean, rstd;
      group_stats(a, [&](int e) { return pivots[ch + e]; }, [&](int e) { return total[ch + e]; }, &mean, &rstd);
      if (lane == 0) {
        grp[g] = make_float2(mean, rstd);
        if (rank == 0) {
          a.mean[st.n * a.G + g0 + g] = mean;
          a.rstd[st.n * a.G + g0 + g] = rstd;
        }
      }
    }
  }
  __syncthreads();
  if (st.on) {
    float k1[V], k2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int gs = (st.v * V + i) / a.cpg;
      const float2 t = grp[gs];
      if (BWD) {
        const float rs = __ldg(a.rstd + st.n * a.G + g0 + gs);
        k2[i] = -rs * rs * t.y;
        k1[i] = -rs * t.x;
      } else {
        m[i] = t.x;
        w[i] *= t.y;
        k1[i] = k2[i] = 0.f;
      }
    }
    int k = 0;
    for (int r = st.r0 + st.row; r < st.r1; r += st.lanes, ++k) {
      float f[V], d[V];
      read_piece<T, V>(xs + (size_t)k * kThreads * PB, f);
      if constexpr (BWD) read_piece<T, V>(ds + (size_t)k * kThreads * PB, d);
      apply<V, ACT, BWD>(f, d, m, w, b, k1, k2);
      write_piece<T, V>(out + (long long)r * a.C + c, f);
    }
  }
  cluster_wait();                                  // no CTA leaves while its sums are being read
}

// In passes. A block takes `rows` rows of one sample and up to kThreads pieces of a row.
template <int V>
struct Span {
  int n, chunk, c, v0, nv, v, row, lanes, r0, r1;
  bool on;
  // the first pass runs forwards through the tensor, the second backwards
  __device__ __forceinline__ Span(const Args& a, bool back) {
    const long long id = back ? (long long)gridDim.x - 1 - blockIdx.x : blockIdx.x;
    chunk = (int)(id % a.chunks);
    n = (int)(id / a.chunks);
    v0 = blockIdx.y * a.cols;
    nv = min(a.cols, a.C / V - v0);
    lanes = kThreads / nv;
    row = (int)threadIdx.x / nv;
    v = (int)threadIdx.x - row * nv;
    on = row < lanes;
    c = (v0 + v) * V;
    r0 = chunk * a.rows;
    r1 = min(a.S, r0 + a.rows);
  }
};

// Rows that a thread has in flight in the passes, in shared memory, as copies that need no
// registers: 64 KB a block. (With two to four rows in registers instead the sums of 2 x 65536 x 512
// took 31 us forward and 78 backward.)
template <bool BWD>
constexpr int kAhead = BWD ? 4 : 8;
template <typename T, int V, bool BWD>
constexpr int kRingBytes = V > 1 ? kAhead<BWD> * (BWD ? 2 : 1) * kThreads * 16 : 0;

// Calls f(x's values, dy's values) for `left` pieces, the first at px and pd, step_x and step_d apart.
template <typename T, int V, bool BWD, typename F>
__device__ __forceinline__ void for_pieces(char* ring, const T* px, const T* pd, long long step_x, long long step_d,
                                           int left, F f) {
  if constexpr (V > 1) {
    constexpr int K = kAhead<BWD>, SLOT = (BWD ? 2 : 1) * kThreads * 16;
    char* mine = ring + threadIdx.x * 16;
    int asked = 0;
    auto ask = [&](int slot) {
      if (asked < left) {
        fetch_piece<T, V>(mine + slot * SLOT, px);
        if (BWD) fetch_piece<T, V>(mine + slot * SLOT + kThreads * 16, pd);
        px += step_x;
        pd += step_d;
        ++asked;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < K; ++k) ask(k);
    for (int i = 0; i < left;) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (i < left) {
          asm volatile("cp.async.wait_group %0;" ::"n"(K - 1) : "memory");
          float x[V], d[V];
          read_piece<T, V>(mine + k * SLOT, x);
          if constexpr (BWD) read_piece<T, V>(mine + k * SLOT + kThreads * 16, d);
          ask(k);
          f(x, d);
          ++i;
        }
      }
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < left; ++i) {
      float x[V], d[V];
      x[0] = to_f32(px[i * step_x]);
      if constexpr (BWD) d[0] = to_f32(pd[i * step_d]);
      f(x, d);
    }
  }
}

template <typename T, int V, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) sums_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) char gn_smem[];
  float2* sums = (float2*)(gn_smem + kRingBytes<T, V, BWD>);
  float2* red = sums + a.cols * V;
  grid_next();
  const Span<V> st(a, false);
  const T* x = (const T*)a.x + st.n * a.sb;
  const T* dy = (const T*)a.dy + (long long)st.n * a.S * a.C;
  float w[V], b[V], m[V], s[V] = {}, q[V] = {};
  if (st.on) {
    if constexpr (BWD) {
      load_channels<V>(a.w, st.c, 1.f, w);
      load_channels<V>(a.b, st.c, 0.f, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = st.n * a.G + (st.c + i) / a.cpg;
        m[i] = __ldg(a.mean + g);
        w[i] *= __ldg(a.rstd + g);
      }
    } else {
      load_pivots<T, V>(x + st.c, a.ss, a.S, m);
    }
    const long long row = st.r0 + st.row;
    for_pieces<T, V, BWD>(gn_smem, x + row * a.ss + st.c, dy + row * a.C + st.c, st.lanes * a.ss, (long long)st.lanes * a.C,
                          (st.r1 - st.r0 - st.row + st.lanes - 1) / st.lanes,
                          [&](float (&f)[V], float (&d)[V]) { add_sums<V, ACT, BWD>(f, d, m, w, b, s, q); });
  }
  turn_back<V, ACT, BWD>(s, q);
  block_sums<V>(s, q, st.nv, red, sums);
  __syncthreads();
  float2* to = a.part + ((long long)st.n * a.chunks + st.chunk) * a.C + st.v0 * V;
  for (int e = threadIdx.x; e < st.nv * V; e += kThreads) to[e] = sums[e];
}

// The chunks' sums of a group's channels, in order, and what follows from them; a block a (sample,
// group). Threads side by side take channels side by side, the others further chunks.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) char gn_smem[];
  float2* chan = (float2*)gn_smem;                 // [cpg]
  __shared__ float2 parts[kThreads];
  __shared__ float pivots[BWD ? 1 : kThreads];
  grid_next();
  const int n = blockIdx.x / a.G, g = blockIdx.x - n * a.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the pivots, which no kernel of this call writes, fetched ahead
  const auto pivot = [&](int e) {                  // (S = 0: x has no element to look at)
    float m[1] = {0.f};
    if (a.S > 0) load_pivots<T, 1>((const T*)a.x + n * a.sb + (long long)g * a.cpg + e, a.ss, a.S, m);
    return m[0];
  };
  const float first = !BWD && threadIdx.x < a.cpg ? pivot(threadIdx.x) : 0.f;
  grid_wait();
  const float2* from = a.part + (long long)n * a.chunks * a.C + (long long)g * a.cpg;
  if (!BWD) pivots[threadIdx.x] = first;
  // (without rows the sums are 0 and rstd is infinite where eps is 0)
  const float rs = BWD && a.S > 0 ? __ldg(a.rstd + blockIdx.x) : 1.f;
  for (int c0 = 0; c0 < a.cpg; c0 += kThreads) {
    const int cols = min(kThreads, a.cpg - c0), per = kThreads / cols;
    const int sub = (int)threadIdx.x / cols, c = (int)threadIdx.x - sub * cols;
    float2 t = make_float2(0.f, 0.f);
    if (sub < per)
#pragma unroll 8
      for (int k = sub; k < a.chunks; k += per) {
        const float2 x = from[(long long)k * a.C + c0 + c];
        t.x += x.x;
        t.y += x.y;
      }
    parts[threadIdx.x] = t;
    __syncthreads();
    if (sub == 0) {
      for (int p = 1; p < per; ++p) {
        t.x += parts[p * cols + c].x;
        t.y += parts[p * cols + c].y;
      }
      chan[c0 + c] = make_float2(t.x, t.y * rs);
    }
    __syncthreads();
  }
  if constexpr (BWD) {
    float c1 = 0.f, c2 = 0.f;
    for (int c = threadIdx.x; c < a.cpg; c += kThreads) {
      const float2 t = chan[c];
      a.chan[(long long)n * a.C + (long long)g * a.cpg + c] = t;
      const float wc = a.w ? __ldg(a.w + (long long)g * a.cpg + c) : 1.f;
      c1 = fmaf(wc, t.x, c1);
      c2 = fmaf(wc, t.y, c2);
    }
    c1 = warp_sum(c1);
    c2 = warp_sum(c2);
    if (lane == 0) parts[warp] = make_float2(c1, c2);
    __syncthreads();
    if (threadIdx.x == 0) {
      float2 t = make_float2(0.f, 0.f);
      for (int k = 0; k < kWarps; ++k) {
        t.x += parts[k].x;
        t.y += parts[k].y;
      }
      const float m = (float)a.S * (float)a.cpg;
      a.coef[blockIdx.x] = make_float2(t.x / m, t.y / m);
    }
  } else if (warp == 0) {
    float mean, rstd;
    group_stats(a, [&](int e) { return e < kThreads ? pivots[e] : pivot(e); }, [&](int e) { return chan[e]; }, &mean,
                &rstd);
    if (lane == 0) {
      a.mean[blockIdx.x] = mean;
      a.rstd[blockIdx.x] = rstd;
    }
  }
}

template <typename T, int V, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) apply_kernel(const __grid_constant__ Args a) {
  grid_next();
  grid_wait();
  const Span<V> st(a, true);
  if (!st.on) return;
  float m[V], w[V], b[V], k1[V], k2[V];
  load_channels<V>(a.w, st.c, 1.f, w);
  load_channels<V>(a.b, st.c, 0.f, b);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int g = st.n * a.G + (st.c + i) / a.cpg;
    const float rs = a.rstd[g];
    m[i] = a.mean[g];
    w[i] *= rs;
    k1[i] = k2[i] = 0.f;
    if (BWD) {
      const float2 t = a.coef[g];
      k2[i] = -rs * rs * t.y;
      k1[i] = -rs * t.x;
    }
  }
  // backwards within the chunk too
  extern __shared__ __align__(16) char gn_smem[];
  const int left = (st.r1 - st.r0 - st.row + st.lanes - 1) / st.lanes;
  const long long step = (long long)st.lanes * a.C;
  const long long row = st.r0 + st.row + (long long)(left - 1) * st.lanes;
  const long long cont = (long long)st.n * a.S * a.C + row * a.C + st.c;
  T* out = (T*)a.out + cont;
  for_pieces<T, V, BWD>(gn_smem, (const T*)a.x + st.n * a.sb + row * a.ss + st.c, (const T*)a.dy + cont,
                        -st.lanes * a.ss, -step, left, [&](float (&f)[V], float (&d)[V]) {
                          apply<V, ACT, BWD>(f, d, m, w, b, k1, k2);
                          write_piece<T, V>(out, f);
                          out -= step;
                        });
}

// dw and db: the samples' channel sums, in order.
__global__ void __launch_bounds__(256) weight_grad_kernel(const __grid_constant__ Args a) {
  grid_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.C) return;
  float2 t = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int n = 0; n < a.N; ++n) {
    const float2 x = a.chan[(long long)n * a.C + c];
    t.x += x.x;
    t.y += x.y;
  }
  if (a.db) a.db[c] = t.x;
  if (a.dw) a.dw[c] = t.y;
}

// ---- host ---------------------------------------------------------------------------------

int lcm(int a, int b) {
  int x = a, y = b;
  while (y) {
    const int r = x % y;
    x = y;
    y = r;
  }
  return a / x * b;
}

// Entries that block_sums needs where rows of `all` pieces are taken `nv` at a time (the last time
// fewer, which may need more).
long long sum_room(int all, int nv, int V) {
  const int last = all % nv ? all % nv : nv;
  return std::max((long long)sum_rows(nv) * nv, (long long)sum_rows(last) * last) * V;
}

// How a call is cut. resident: clusters of `cluster` CTAs; else chunks of rows.
struct Plan {
  bool resident;
  int slab, slabs, cluster, rows, pieces, smem;
  int chunks, cols;
};

// How a call is cut, by what both ways measured (us on the GPU).
// Resident: among the cuts that fit, the one of the least count: each round of the chip's CTAs takes 6
// (backward 9) and what its bytes take at 44 GB/s an SM, a third more where a row of a slab is under 64
// bytes, and 1 more for each doubling of the cluster (clusters of 8 and 16 wait long for their places: never).
// Resident or in passes: instructions for each element are what either takes next to its latency, so a round
// takes 6.7 and 0.15 for each 1000 elements of an SM (backward 7.8 and 0.26), the passes 11.4 and 1.03 for
// each million elements (15.3 and 1.54). Resident / in passes, the chosen one with a star:
//   bf16        4 x 1024 x 512   4 x 4096 x 512   8 x 1024 x 1280   8 x 4096 x 320   8 x 4096 x 512
//   forward     9.4* / 13.3      15.5* / 21.1     18.2* / 23.1      19.2* / 21.5     29.7 / 26.7*
//   backward    13.3* / 19.5     30.6 / 29.7*     39.4 / 32.1*      39.6 / 29.3*     58 / 40*
//   fp32 4 x 4096 x 512: 24.2 / 21.4* and 43 / 32*; bf16 2 x 4096 x 320: 12.4* / 13.2 and 20.1* / 18.3
Plan make_plan(int N, int S, int C, int G, int V, int e, bool bwd) {
  Plan p = {};
  const int cpg = C / G;
  double best = 1e300, resident = 0;
  const int unit = S > 0 ? lcm(cpg, V) : C + 1;      // slabs are whole groups and whole pieces
  for (int slab = unit; slab <= C && slab <= 2048 && slab / V <= kThreads; slab += slab < unit * 4 ? unit : slab) {
    if (slab * e < 32 && slab + unit <= C) continue;
    if (slab * e > 512 && slab > unit) break;
    const int nv = slab / V, lanes = kThreads / nv, slabs = ceil_div(C, slab);
    for (int cl = 1; cl <= 4; cl *= 2) {
      const int rows = ceil_div(S, cl), pieces = ceil_div(rows, lanes);
      const long long bytes = (long long)pieces * kThreads * V * e * (bwd ? 2 : 1);
      const long long smem = (long long)round_up_to(bytes, 16) +
                             (sum_room(C / V, nv, V) + 2 * slab + slab / cpg + (bwd ? 0 : (slab + 1) / 2)) *
                                 (long long)sizeof(float2);
      if (smem > kMaxShared) continue;
      const int held = smem + 1024 <= kMaxShared / 2 ? 2 : 1;
      const long long ctas = (long long)N * slabs * cl, rounds = ceil_div<long long>(ctas, kChip * held);
      const double moved = (double)rows * slab * e * (bwd ? 3 : 2) * std::min<double>(held, std::max(1.0, (double)ctas / kChip));
      const double t = rounds * ((bwd ? 9 : 6) + moved * (slab * e < 64 ? 1.33 : 1.0) / 44e3) + (cl == 4 ? 2 : cl - 1);
      if (t < best) {
        best = t;
        resident = rounds * ((bwd ? 7.8 : 6.7) + moved / ((bwd ? 3 : 2) * e) * (bwd ? 0.26e-3 : 0.15e-3));
        p.resident = true;
        p.slab = slab;
        p.slabs = slabs;
        p.cluster = cl;
        p.rows = rows;
        p.pieces = pieces;
        p.smem = (int)smem;
      }
    }
  }
  p.resident = p.resident && resident <= (bwd ? 15.3 : 11.4) + (double)N * S * C * (bwd ? 1.54e-6 : 1.03e-6);
  if (p.resident) return p;
  p = {};
  const int nv = C / V;
  p.cols = std::min(nv, kThreads);
  const int lanes = kThreads / p.cols;
  // chunks: the two blocks that an SM holds, each with rows enough to pay for its sums
  const long long blocks = 2ll * kChip;
  const long long want = std::max<long long>(1, blocks / std::max<long long>(1, (long long)N * ceil_div(nv, p.cols)));
  p.rows = std::max(8 * lanes, (int)ceil_div<long long>(S, want));
  p.chunks = ceil_div(S, p.rows);
  p.smem = (int)(sum_room(nv, p.cols, V) + p.cols * V) * (int)sizeof(float2);
  return p;
}

// The widest need over both piece widths and directions.
size_t workspace_bytes_of(long long N, long long S, long long C, int G, size_t* part, size_t* chan, size_t* coef) {
  size_t chunks = 0;
  for (int V : {1, 4, 8})
    if (C % V == 0)
      for (int e : {2, 4})
        for (bool bwd : {false, true}) chunks = std::max<size_t>(chunks, make_plan((int)N, (int)S, (int)C, G, V, e, bwd).chunks);
  *part = 0;
  *chan = round_up_to(*part + (size_t)N * chunks * C * sizeof(float2), 256);
  *coef = round_up_to(*chan + (size_t)N * C * sizeof(float2), 256);
  return round_up_to(std::max<size_t>(*coef + (size_t)N * G * sizeof(float2), 256), 256);
}

bool sizes_ok(long long N, long long S, long long C, int G) {
  return N >= 0 && S >= 0 && C >= 1 && G >= 1 && C % G == 0 && C <= (1 << 18) && C / G <= 4096 && N < (1ll << 24) &&
         S < (1ll << 31) - 65536 && N * G < (1ll << 31) - 256 && N * S < (1ll << 31) - 65536 &&
         N * S <= (1ll << 42) / C;
}

template <typename T, int V, int ACT, bool BWD>
dash_status_t launch(Args a, cudaStream_t stream) {
  const Plan p = make_plan(a.N, a.S, a.C, a.G, V, sizeof(T), BWD);
  a.slab = p.slab;
  a.slabs = p.slabs;
  a.rows = p.rows;
  a.chunks = p.chunks;
  a.cols = p.cols;
  if (a.N == 0) {
    // no sample: dw and db are zeros
  } else if (p.resident) {
    const auto kernel = resident_kernel<T, V, ACT, BWD>;
    DASH_TRY(allow_shared((const void*)kernel, p.smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.N * p.slabs * p.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    DASH_TRY(cudaLaunchKernelEx(&cfg, kernel, a, p.pieces));
  } else {
    const dim3 grid((unsigned)a.N * p.chunks, ceil_div(a.C / V, p.cols));
    if (grid.x > 0) {
      const int smem = p.smem + kRingBytes<T, V, BWD>;
      DASH_TRY(allow_shared((const void*)sums_kernel<T, V, ACT, BWD>, smem));
      sums_kernel<T, V, ACT, BWD><<<grid, kThreads, smem, stream>>>(a);
      DASH_TRY(cudaGetLastError());
    }
    DASH_TRY(launch_after(join_kernel<T, BWD>, dim3((unsigned)a.N * a.G), kThreads, a.cpg * sizeof(float2), stream, a));
    if (grid.x > 0) {
      DASH_TRY(allow_shared((const void*)apply_kernel<T, V, ACT, BWD>, kRingBytes<T, V, BWD>));
      DASH_TRY(launch_after(apply_kernel<T, V, ACT, BWD>, grid, kThreads, kRingBytes<T, V, BWD>, stream, a));
    }
  }
  if (BWD && (a.dw || a.db))
    DASH_TRY(launch_after(weight_grad_kernel, dim3(ceil_div(a.C, 256)), 256, 0, stream, a));
  return DASH_OK;
}

template <typename T, bool BWD>
dash_status_t by_act(const Args& a, int act, bool vec, cudaStream_t stream) {
  if (vec) return act == SILU ? launch<T, kVec<T>, SILU, BWD>(a, stream) : launch<T, kVec<T>, NONE, BWD>(a, stream);
  return act == SILU ? launch<T, 1, SILU, BWD>(a, stream) : launch<T, 1, NONE, BWD>(a, stream);
}

template <bool BWD>
dash_status_t by_type(const Args& a, int act, int dtype, cudaStream_t stream) {
  const int e = dtype == DASH_FP32 ? 4 : 2, v = 16 / e;
  // 16-byte pieces where every row is made of them
  bool vec = a.C % v == 0 && a.ss % v == 0 && a.sb % v == 0;
  for (const void* p : {a.x, a.dy, (const void*)a.out}) vec = vec && is_aligned(p, 16);
  if (dtype == DASH_BF16) return by_act<__nv_bfloat16, BWD>(a, act, vec, stream);
  if (dtype == DASH_FP16) return by_act<__half, BWD>(a, act, vec, stream);
  return by_act<float, BWD>(a, act, vec, stream);
}

dash_status_t check(const void* x, const float* w, const float* b, const float* mean, const float* rstd,
                    const void* out, void* workspace, size_t workspace_bytes, long long N, long long S, long long C,
                    int G, const long long* xs, float eps, int act, int dtype, Args* a) {
  if (N < 0 || S < 0 || C < 1 || G < 1 || C % G || !(eps >= 0.f) || !xs) return DASH_ERR_INVALID_ARG;
  if (act != NONE && act != SILU) return DASH_ERR_INVALID_ARG;
  if (dtype != DASH_BF16 && dtype != DASH_FP16 && dtype != DASH_FP32) return DASH_ERR_INVALID_ARG;
  if (!sizes_ok(N, S, C, G)) return DASH_ERR_UNSUPPORTED;
  if (xs[0] < 0 || xs[1] < 0 || xs[0] > (1ll << 40) || xs[1] > (1ll << 40)) return DASH_ERR_UNSUPPORTED;
  if (N * S > 0 && (!x || !out)) return DASH_ERR_INVALID_ARG;
  if (N > 0 && (!mean || !rstd)) return DASH_ERR_INVALID_ARG;
  const int e = dtype == DASH_FP32 ? 4 : 2;
  if (!is_aligned(x, e) || !is_aligned(out, e)) return DASH_ERR_INVALID_ARG;
  for (const float* p : {w, b, mean, rstd})
    if (!is_aligned(p, 4)) return DASH_ERR_INVALID_ARG;
  if (!workspace || !is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  size_t part, chan, coef;
  if (workspace_bytes < workspace_bytes_of(N, S, C, G, &part, &chan, &coef)) return DASH_ERR_WORKSPACE_TOO_SMALL;
  char* ws = (char*)workspace;
  *a = {};
  a->x = x;
  a->out = const_cast<void*>(out);
  a->w = w;
  a->b = b;
  a->mean = const_cast<float*>(mean);
  a->rstd = const_cast<float*>(rstd);
  a->part = (float2*)(ws + part);
  a->chan = (float2*)(ws + chan);
  a->coef = (float2*)(ws + coef);
  a->sb = xs[0];
  a->ss = xs[1];
  a->N = (int)N;
  a->S = (int)S;
  a->C = (int)C;
  a->G = G;
  a->cpg = (int)(C / G);
  a->eps = eps;
  return DASH_OK;
}

}  // namespace

extern "C" {

size_t dash_group_norm_workspace_size(long long N, long long S, long long C, int G) {
  if (!sizes_ok(N, S, C, G)) return 0;
  size_t part, chan, coef;
  return workspace_bytes_of(N, S, C, G, &part, &chan, &coef);
}

dash_status_t dash_group_norm_fwd(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd,
                                  void* workspace, size_t workspace_bytes, long long N, long long S, long long C,
                                  int G, const long long* x_strides, float eps, int act, int dtype,
                                  cudaStream_t stream) {
  Args a;
  const dash_status_t st = check(x, w, b, mean, rstd, y, workspace, workspace_bytes, N, S, C, G, x_strides, eps, act,
                                 dtype, &a);
  if (st != DASH_OK) return st;
  if (N == 0) return DASH_OK;
  return by_type<false>(a, act, dtype, stream);
}

dash_status_t dash_group_norm_bwd(const void* dy, const void* x, const float* w, const float* b, const float* mean,
                                  const float* rstd, void* dx, float* dw, float* db, void* workspace,
                                  size_t workspace_bytes, long long N, long long S, long long C, int G,
                                  const long long* x_strides, int act, int dtype, cudaStream_t stream) {
  Args a;
  const dash_status_t st = check(x, w, b, mean, rstd, dx, workspace, workspace_bytes, N, S, C, G, x_strides, 0.f, act,
                                 dtype, &a);
  if (st != DASH_OK) return st;
  if ((N * S > 0 && !dy) || !is_aligned(dy, dtype == DASH_FP32 ? 4 : 2) || !is_aligned(dw, 4) || !is_aligned(db, 4))
    return DASH_ERR_INVALID_ARG;
  a.dy = dy;
  a.dw = dw;
  a.db = db;
  return by_type<true>(a, act, dtype, stream);
}

}  // extern "C"
