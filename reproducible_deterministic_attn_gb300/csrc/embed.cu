// Token embedding (dash_embed_fwd) and its gradient by sorted tokens (dash_embed_bwd).
//
// The forward is a gather of rows: one load and one store of 16 bytes a thread and four rows
// in flight, bound by HBM. The gradient has four launches:
//   embed_sort  one cluster of 8 CTAs sorts the tokens by id: a stable counting sort by
//               digits of at most 9 bits, so two passes up to 2^18 ids. Each warp counts a
//               run of tokens of its own, so ranks within a digit follow the token order
//               without atomics; the CTAs' counts meet in distributed shared memory. It is
//               bound by latency (some 20 k cycles).
//   embed_zero  zeroes the whole table meanwhile: it starts beside the sort and does not wait
//               for it; the rows of ids that occur are then stored over the zeroes.
//   embed_rows  runs of 32 sorted places times column tiles: an id's rows are added in
//               order in registers; ids that lie within one run are stored, the parts of
//               those that cross runs go to the workspace.
//   embed_join  adds the parts of the ids that cross runs, in order.
// Measured at 16384 tokens x 2048 bf16, 65536 ids falling off as 1/rank: lookup 20 us (134 MB),
// sort 18, zero 37 (268 MB, beside the sort), rows 17, join 9 us, the gradient together 63 us
// (335 MB would take 49). Runs of 8 places instead of 32: 75 us, the join's lists grow. 65536
// and 262144 tokens: sort 49 and 158, rows 66 and 200, join 14 and 49 us, together 146 and 415 (79
// and 198 by their bytes).
#include <cooperative_groups.h>

#include <algorithm>

#include "dash_train.h"
#include "host_common.h"
#include "train_common.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace dash;
using namespace dash::train;

constexpr int kRun = 32;                // sorted places a run
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kAheadStrips = 4;         // strips of 32 tokens a warp has in flight

// ---- forward ------------------------------------------------------------------------------

constexpr int kFwdThreads = 256;
constexpr int kFwdRows = 4;             // rows a team of threads has in flight

template <typename T, int VEC>
__global__ void __launch_bounds__(kFwdThreads)
    embed_fwd_kernel(const T* table, const void* ids, T* out, int* status, long long n, long long V, int D,
                     long long ld_table, long long ld_out, float scale, int id_bits, int tx) {
  const int x = threadIdx.x % tx, y = threadIdx.x / tx, ty = kFwdThreads / tx;
  const long long row0 = (long long)blockIdx.x * ty * kFwdRows + y;
  long long id[kFwdRows];
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) {
    const long long row = row0 + r * ty;
    id[r] = row < n ? load_index(ids, row, id_bits) : -2;
    if (row < n && (id[r] < 0 || id[r] >= V)) {
      id[r] = -1;
      if (x == 0 && status) *status = kStatusBounds;
    }
  }
  for (int c = x * VEC; c < D; c += tx * VEC) {
    Vec<T, VEC> v[kFwdRows];
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      v[r] = {};
      if (id[r] >= 0) v[r] = load_vec<T, VEC>(table + id[r] * ld_table + c);
    }
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      if (id[r] == -2) continue;
      if (id[r] < 0 || scale != 1.f) {
        float f[VEC];
        unpack<T, VEC>(v[r], f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = id[r] < 0 ? NAN : f[i] * scale;
        v[r] = pack<T, VEC>(f);
      }
      store_vec<T, VEC>(out + (row0 + r * ty) * ld_out + c, v[r]);
    }
  }
}

// ---- the sort -----------------------------------------------------------------------------

struct SortArgs {
  const void* ids;
  int id_bits;
  long long T, V, padding_idx;
  int passes, digit_bits;
  int* header;
  uint2* sorted[2];           // (id, token); the last pass writes index (passes - 1) & 1
};

// Zeroes n bytes at p, both even. The kernel before it is this call's sort, which starts only
// when all earlier work is done, so the table may be written at once. Its first block then
// waits for the sort, so that what waits for this kernel waits for both.
constexpr int kZeroThreads = 256;
constexpr size_t kZeroBytes = 1 << 16;  // of one block
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(char* p, size_t n) {
  grid_next();
  const size_t from = blockIdx.x * kZeroBytes;
  p += from;
  n = min(kZeroBytes, n - from);
  const size_t head = min(n, (size_t)(-(intptr_t)p & 15)), body = (n - head) / 16, tail = n - head - body * 16;
#pragma unroll 8
  for (size_t i = threadIdx.x; i < body; i += kZeroThreads)
    reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < head / 2) reinterpret_cast<uint16_t*>(p)[threadIdx.x] = 0;
  if (threadIdx.x < tail / 2) reinterpret_cast<uint16_t*>(p + head + body * 16)[threadIdx.x] = 0;
  if (blockIdx.x == 0) grid_wait();
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads)
    embed_sort_kernel(const SortArgs a) {
  extern __shared__ unsigned sort_smem[];
  const int bins = 1 << a.digit_bits;
  unsigned* hist = sort_smem;                       // [warps][bins]
  unsigned* cta_total = hist + kSortWarps * bins;   // [bins]
  unsigned* base = cta_total + bins;                // [bins]
  __shared__ unsigned warp_sums[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned lt = (1u << lane) - 1;

  grid_next();
  if (rank == 0 && threadIdx.x < kWsHeaderBytes / 4) a.header[threadIdx.x] = 0;

  // this warp's run of whole 32-token strips
  const long long strips = (a.T + 31) / 32;
  const long long per_warp = (strips + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps);
  const long long first = ((long long)rank * kSortWarps + warp) * per_warp;
  const long long last = min(strips, first + per_warp);
  unsigned* mine = hist + warp * bins;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit_bits;
    const uint2* src = a.sorted[(pass + 1) & 1];
    uint2* dst = a.sorted[pass & 1];
    auto pair_at = [&](long long t) -> uint2 {
      if (pass > 0) return __ldcg(src + t);
      const long long id = load_index(a.ids, t, a.id_bits);
      return make_uint2(id < 0 || id >= a.V || id == a.padding_idx ? (unsigned)a.V : (unsigned)id, (unsigned)t);
    };
    auto load_strips = [&](long long s, uint2 (&pair)[kAheadStrips]) {
#pragma unroll
      for (int k = 0; k < kAheadStrips; ++k) {
        const long long t = (s + k) * 32 + lane;
        pair[k] = s + k < last && t < a.T ? pair_at(t) : make_uint2(0, 0);
      }
    };
    for (int d = lane; d < bins; d += 32) mine[d] = 0;
    __syncwarp();
    uint2 pair[kAheadStrips];
    for (long long s = first; s < last; s += kAheadStrips) {
      load_strips(s, pair);
#pragma unroll
      for (int k = 0; k < kAheadStrips; ++k) {
        const bool in = s + k < last && (s + k) * 32 + lane < a.T;
        const unsigned live = __ballot_sync(0xffffffffu, in);
        if (in) {
          const unsigned d = (pair[k].x >> shift) & (bins - 1);
          const unsigned peers = __match_any_sync(live, d);
          if ((peers & lt) == 0) mine[d] += __popc(peers);
        }
        __syncwarp();
      }
    }
    __syncthreads();
    // counts -> offsets of the warps within the CTA, and the CTA's totals (bins <= threads)
    const int d = threadIdx.x;
    if (d < bins) {
      unsigned run = 0;
#pragma unroll 1
      for (int w0 = 0; w0 < kSortWarps; w0 += 8) {
        unsigned c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = hist[(w0 + w) * bins + d];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          hist[(w0 + w) * bins + d] = run;
          run += c[w];
        }
      }
      cta_total[d] = run;
    }
    cluster.sync();
    // offset of each digit over all CTAs
    unsigned lower = 0, total = 0;
    if (d < bins) {
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        const unsigned v = *cluster.map_shared_rank(cta_total + d, c);
        if (c < rank) lower += v;
        total += v;
      }
    }
    // After the last pass nobody reads the sorted array here: a CTA only has to stay until the
    // others have read its totals, so they say so now and wait at the end.
    const bool last_pass = pass + 1 == a.passes;
    if (last_pass) cluster.barrier_arrive();
    unsigned scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0u);
    if (d < bins) base[d] = before + scan - total + lower;
    __syncthreads();
    for (long long s = first; s < last; s += kAheadStrips) {
      if (last - first > kAheadStrips) load_strips(s, pair);   // else they are still there
#pragma unroll
      for (int k = 0; k < kAheadStrips; ++k) {
        const long long t = (s + k) * 32 + lane;
        const bool in = s + k < last && t < a.T;
        const unsigned live = __ballot_sync(0xffffffffu, in);
        unsigned dg = 0, peers = 0;
        if (in) {
          dg = (pair[k].x >> shift) & (bins - 1);
          peers = __match_any_sync(live, dg);
          // one store for both: an SM takes some cycles for each place of a scattered store,
          // which is most of what a pass costs
          dst[base[dg] + mine[dg] + __popc(peers & lt)] = pair[k];
          if (pass == 0 && pair[k].x >= a.V) {
            const long long id = load_index(a.ids, t, a.id_bits);
            if (id < 0 || id >= a.V) report_index(a.header, CHK_TOKEN_ID, t, id, a.V);
          }
        }
        __syncwarp();
        if (in && (peers & lt) == 0) mine[dg] += __popc(peers);
        __syncwarp();
      }
    }
    if (last_pass) cluster.barrier_wait();
    else cluster.sync();                // the totals have been read; the sorted array is visible
  }
}

// ---- the rows -----------------------------------------------------------------------------

struct RowArgs {
  const uint2* sorted;        // (id, token) by id
  long long T, V;
  int D;
  long long ld_dout;
  float scale;
  int accumulate;
  float* part;                // [runs][2][Dp]: 0 = of an id begun in an earlier run, 1 = of one
  int Dp;                     //     that goes on in the next
  int tx, col_tiles;
  long long runs;
};

constexpr int kRowThreads = 128;

// A thread's columns of a row: VEC consecutive ones in whole 16-byte pieces, or four ones that
// lie tx apart (STRIDED: rows that are no whole pieces), of which `n` are there.
constexpr int kStridedCols = 4;
template <typename T, int N, bool STRIDED>
struct Cols;
template <typename T, int N>
struct Cols<T, N, false> {
  Vec<T, N> v;
  __device__ __forceinline__ void load(const T* p, int, int) { v = load_vec<T, N>(p); }
  __device__ __forceinline__ void get(float (&f)[N]) const { unpack<T, N>(v, f); }
  __device__ __forceinline__ void put(T* p, const float (&f)[N], int, int) const { store_f32<T, N>(p, f); }
};
template <typename T, int N>
struct Cols<T, N, true> {
  T v[N];
  __device__ __forceinline__ void load(const T* p, int tx, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? p[i * tx] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(v[i]);
  }
  __device__ __forceinline__ void put(T* p, const float (&f)[N], int tx, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i * tx] = from_f32<T>(f[i]);
  }
};

template <typename TO, int N, bool STRIDED>
__device__ __forceinline__ void put_cols(TO* dst, const float (&acc)[N], float scale, int accumulate, int tx,
                                         int n) {
  Cols<TO, N, STRIDED> c;
  float x[N];
  if (accumulate) {
    c.load(dst, tx, n);
    c.get(x);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(acc[i], scale, x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = acc[i] * scale;
  }
  c.put(dst, x, tx, n);
}

template <typename TI, typename TO, bool STRIDED>
__global__ void __launch_bounds__(kRowThreads)
    embed_rows_kernel(const TI* dout, TO* dtable, const RowArgs a) {
  constexpr int N = STRIDED ? kStridedCols : 16 / sizeof(TI);
  const int x = threadIdx.x % a.tx, y = threadIdx.x / a.tx, ty = kRowThreads / a.tx;
  const int tile = a.tx * N;                       // columns a team of tx threads covers
  const int off = STRIDED ? x : x * N;
  // the places of the block's runs, with the one before and the one after each
  extern __shared__ uint2 rows_smem[];
  grid_next();
  grid_wait();
  const long long run0 = (blockIdx.x / a.col_tiles) * (long long)ty;
  for (int i = threadIdx.x; i < ty * (kRun + 2); i += kRowThreads) {
    const long long at = (run0 + i / (kRun + 2)) * kRun + i % (kRun + 2) - 1;
    rows_smem[i] = at >= 0 && at < a.T ? a.sorted[at] : make_uint2(0xffffffffu, 0);
  }
  __syncthreads();
  const long long run = run0 + y;
  const int c0 = (int)(blockIdx.x % a.col_tiles) * tile, col = c0 + off;
  if (run >= a.runs || col >= a.D) return;
  const int nc = STRIDED ? min(N, (a.D - col + a.tx - 1) / a.tx) : N;   // columns that are there
  const int n = (int)min((long long)kRun, a.T - run * kRun);
  const unsigned V = (unsigned)a.V;
  const uint2* sorted = rows_smem + y * (kRun + 2) + 1;
  unsigned key = sorted[0].x;
  bool begun = sorted[-1].x == key;
  float acc[N] = {};
  constexpr int U = 8;                             // rows in flight a thread (16: 17 -> 23 us for 16384 x 2048)
#pragma unroll 1
  for (int p = 0; p < n && key < V; p += U) {
    Cols<TI, N, STRIDED> v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      v[i] = {};
      if (p + i < n) v[i].load(dout + sorted[p + i].y * a.ld_dout + col, a.tx, nc);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (p + i < n && key < V) {
        float f[N];
        v[i].get(f);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += f[k];
        const unsigned next = sorted[p + i + 1].x;
        if (next != key || p + i + 1 == n) {
          if (!begun && next != key) {
            put_cols<TO, N, STRIDED>(dtable + (long long)key * a.D + col, acc, a.scale, a.accumulate, a.tx, nc);
          } else {
            put_cols<float, N, STRIDED>(a.part + (run * 2 + (begun ? 0 : 1)) * a.Dp + col, acc, 1.f, 0, a.tx, nc);
          }
          begun = false;
          key = next;
#pragma unroll
          for (int k = 0; k < N; ++k) acc[k] = 0.f;
        }
      }
    }
  }
}

__device__ __forceinline__ float4 part_at(const RowArgs& a, long long run, int slot, int col) {
  return __ldcg(reinterpret_cast<const float4*>(a.part + (run * 2 + slot) * a.Dp + col));
}
__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}
template <typename TO>
__device__ __forceinline__ void put4(TO* row, const float4& s, int col, const RowArgs& a) {
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < a.D) {
      const float one[1] = {v[i]};
      put_cols<TO, 1, false>(row + col + i, one, a.scale, a.accumulate, 1, 1);
    }
}

// Joins the parts of the ids that cross runs. A block looks at 8 runs, a warp each, and 128
// columns, 4 a thread. Where an id begins that goes on in the next run, the run's warp adds
// the parts of the following runs in order when they are at most kShort; else the 8 warps add
// an eighth of them each, in order, and then the eighths are added in order.
constexpr int kShort = 4;
template <typename TO>
__global__ void __launch_bounds__(256) embed_join_kernel(TO* dtable, const RowArgs a) {
  __shared__ float4 sums[8][32];
  __shared__ unsigned crossing[8];
  __shared__ int follows[8];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = (blockIdx.y * 32 + lane) * 4;
  grid_wait();
  {
    const long long run = (long long)blockIdx.x * 8 + g, p0 = run * kRun;
    // the run's last key, the next one and the one before the run, at once
    unsigned k = 0xffffffffu;
    if (p0 + kRun < a.T) {
      if (lane == 0) k = a.sorted[p0 + kRun - 1].x;
      if (lane == 1) k = a.sorted[p0 + kRun].x;
      if (lane == 2 && run > 0) k = a.sorted[p0 - 1].x;
    }
    const unsigned key = __shfl_sync(0xffffffffu, k, 0);
    const bool cross = key < (unsigned)a.V && __shfl_sync(0xffffffffu, k, 1) == key &&
                       __shfl_sync(0xffffffffu, k, 2) != key;
    int follow = 0;                                // the following runs that start with this id
    if (cross) {
      for (;;) {
        const long long r = run + 1 + follow + lane;
        const unsigned same = __ballot_sync(0xffffffffu, r < a.runs && a.sorted[r * kRun].x == key);
        follow += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        if (same != 0xffffffffu) break;
      }
      if (follow <= kShort && col < a.Dp) {
        float4 s = part_at(a, run, 1, col);
        float4 v[kShort];
#pragma unroll
        for (int r = 0; r < kShort; ++r) v[r] = r < follow ? part_at(a, run + 1 + r, 0, col) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kShort; ++r)
          if (r < follow) add4(s, v[r]);
        put4(dtable + (long long)key * a.D, s, col, a);
      }
    }
    if (lane == 0) {
      crossing[g] = key;
      follows[g] = follow;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    const int follow = follows[j];
    if (follow <= kShort) continue;
    const long long run = (long long)blockIdx.x * 8 + j;
    const int per = (follow + 7) / 8, end = min(follow, (g + 1) * per);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f), head = s;
    if (col < a.Dp) {
      if (g == 0) head = part_at(a, run, 1, col);
#pragma unroll 8
      for (int r = g * per; r < end; ++r) add4(s, part_at(a, run + 1 + r, 0, col));
    }
    sums[g][lane] = s;
    __syncthreads();
    if (g == 0 && col < a.Dp) {
      for (int k = 0; k < 8; ++k) add4(head, sums[k][lane]);
      put4(dtable + (long long)crossing[j] * a.D, head, col, a);
    }
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------------------

size_t elt_bytes(int dtype) { return dtype == DASH_FP32 ? 4 : 2; }

bool sizes_ok(long long T, long long V, int D) {
  const long long lim = (1ll << 31) - 256;
  return T >= 0 && T < lim && V >= 1 && V < lim && D >= 1 && D <= (1 << 20);
}

int pow2_lanes(int need, int most) {
  int t = 1;
  while (t < need && t < most) t *= 2;
  return t;
}

struct Layout {
  size_t sorted0, sorted1, part, total;
  long long runs;
  int Dp;
};

Layout layout(long long T, int D) {
  Layout l;
  size_t at = kWsHeaderBytes;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at = round_up_to(at + bytes, 256);
    return here;
  };
  l.runs = ceil_div<long long>(T, kRun);
  l.Dp = (int)round_up_to(D, 8);
  l.sorted0 = take((size_t)T * sizeof(uint2));
  l.sorted1 = take((size_t)T * sizeof(uint2));
  l.part = take((size_t)l.runs * 2 * l.Dp * 4);
  l.total = at;
  return l;
}

template <typename T>
dash_status_t fwd_typed(const void* table, const void* ids, void* out, int* status, long long n, long long V,
                        int D, long long ldt, long long ldo, float scale, int id_bits, cudaStream_t stream) {
  constexpr int W = 16 / sizeof(T);
  const bool wide = D % W == 0 && ldt % W == 0 && ldo % W == 0 && is_aligned(table, 16) && is_aligned(out, 16);
  const int tx = pow2_lanes(wide ? D / W : D, kFwdThreads);
  const long long blocks = ceil_div<long long>(n, (long long)(kFwdThreads / tx) * kFwdRows);
  if (wide)
    embed_fwd_kernel<T, W><<<(unsigned)blocks, kFwdThreads, 0, stream>>>((const T*)table, ids, (T*)out, status,
                                                                         n, V, D, ldt, ldo, scale, id_bits, tx);
  else
    embed_fwd_kernel<T, 1><<<(unsigned)blocks, kFwdThreads, 0, stream>>>((const T*)table, ids, (T*)out, status,
                                                                         n, V, D, ldt, ldo, scale, id_bits, tx);
  DASH_TRY(cudaGetLastError());
  return DASH_OK;
}

template <typename TI, typename TO>
dash_status_t rows_typed(const void* dout, void* dtable, RowArgs a, cudaStream_t stream) {
  constexpr int W = 16 / sizeof(TI);
  const bool wide = a.D % W == 0 && a.ld_dout % W == 0 && is_aligned(dout, 16) && is_aligned(dtable, 16);
  const int per = wide ? W : kStridedCols;
  a.tx = pow2_lanes(ceil_div(a.D, per), kRowThreads);
  a.col_tiles = ceil_div(a.D, a.tx * per);
  const long long blocks = ceil_div<long long>(a.runs, kRowThreads / a.tx) * a.col_tiles;
  if (blocks >= (1ll << 31)) return DASH_ERR_UNSUPPORTED;
  DASH_TRY(launch_after(wide ? embed_rows_kernel<TI, TO, false> : embed_rows_kernel<TI, TO, true>,
                        dim3((unsigned)blocks), kRowThreads, kRowThreads / a.tx * (kRun + 2) * sizeof(uint2), stream,
                        (const TI*)dout, (TO*)dtable, a));
  if (a.runs > 1)
    DASH_TRY(launch_after(embed_join_kernel<TO>,
                          dim3((unsigned)ceil_div<long long>(a.runs, 8), (unsigned)ceil_div(a.Dp, 128)), 256, 0,
                          stream, (TO*)dtable, a));
  return DASH_OK;
}

bool dtype_ok(int d) { return d == DASH_BF16 || d == DASH_FP16 || d == DASH_FP32; }

}  // namespace

extern "C" {

dash_status_t dash_embed_fwd(const void* table, const void* ids, void* out, int* status,
                             long long T, long long V, int D, long long ld_table, long long ld_out,
                             float scale, int dtype, int id_bits, cudaStream_t stream) {
  if (!table || (T > 0 && (!ids || !out))) return DASH_ERR_INVALID_ARG;
  if (T < 0 || V < 1 || D < 1 || ld_table < D || ld_out < D) return DASH_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (id_bits != 32 && id_bits != 64)) return DASH_ERR_INVALID_ARG;
  if (!sizes_ok(T, V, D) || ld_table > (1ll << 31) || ld_out > (1ll << 31)) return DASH_ERR_UNSUPPORTED;
  if (!is_aligned(table, elt_bytes(dtype)) || !is_aligned(out, elt_bytes(dtype)) ||
      !is_aligned(ids, id_bits / 8) || !is_aligned(status, 4))
    return DASH_ERR_INVALID_ARG;
  if (status) DASH_TRY(cudaMemsetAsync(status, 0, sizeof(int), stream));
  if (T == 0) return DASH_OK;
  switch (dtype) {
    case DASH_BF16:
      return fwd_typed<__nv_bfloat16>(table, ids, out, status, T, V, D, ld_table, ld_out, scale, id_bits, stream);
    case DASH_FP16:
      return fwd_typed<__half>(table, ids, out, status, T, V, D, ld_table, ld_out, scale, id_bits, stream);
    default:
      return fwd_typed<float>(table, ids, out, status, T, V, D, ld_table, ld_out, scale, id_bits, stream);
  }
}

size_t dash_embed_bwd_workspace_size(long long T, long long V, int D) {
  return sizes_ok(T, V, D) ? layout(T, D).total : 0;
}

dash_status_t dash_embed_bwd(const void* dout, const void* ids, void* dtable, void* workspace,
                             size_t workspace_bytes, long long T, long long V, int D,
                             long long ld_dout, float scale, long long padding_idx, int accumulate,
                             int dout_dtype, int dtable_dtype, int id_bits, cudaStream_t stream) {
  if (!dtable || !workspace || (T > 0 && (!dout || !ids))) return DASH_ERR_INVALID_ARG;
  if (T < 0 || V < 1 || D < 1 || ld_dout < D || padding_idx < -1) return DASH_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DASH_ERR_INVALID_ARG;
  if (!dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype) || (id_bits != 32 && id_bits != 64))
    return DASH_ERR_INVALID_ARG;
  if (dtable_dtype != dout_dtype && dtable_dtype != DASH_FP32) return DASH_ERR_UNSUPPORTED;
  if (!sizes_ok(T, V, D) || ld_dout > (1ll << 31)) return DASH_ERR_UNSUPPORTED;
  if (!is_aligned(dout, elt_bytes(dout_dtype)) || !is_aligned(dtable, elt_bytes(dtable_dtype)) ||
      !is_aligned(ids, id_bits / 8) || !is_aligned(workspace, 256))
    return DASH_ERR_INVALID_ARG;
  const Layout l = layout(T, D);
  if (workspace_bytes < l.total) return DASH_ERR_WORKSPACE_TOO_SMALL;
  char* ws = (char*)workspace;
  if (T == 0) {
    DASH_TRY(cudaMemsetAsync(ws, 0, kWsHeaderBytes, stream));
    if (!accumulate) DASH_TRY(cudaMemsetAsync(dtable, 0, (size_t)V * D * elt_bytes(dtable_dtype), stream));
    return DASH_OK;
  }
  SortArgs s;
  s.ids = ids;
  s.id_bits = id_bits;
  s.T = T;
  s.V = V;
  s.padding_idx = padding_idx;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;          // keys 0 .. V (V: left out)
  s.passes = ceil_div(bits, kMaxDigitBits);
  s.digit_bits = ceil_div(bits, s.passes);
  s.header = (int*)ws;
  const size_t table_bytes = (size_t)V * D * elt_bytes(dtable_dtype);
  const size_t zero_blocks = ceil_div<size_t>(table_bytes, kZeroBytes);
  if (zero_blocks >= (1ull << 31)) return DASH_ERR_UNSUPPORTED;
  s.sorted[0] = (uint2*)(ws + l.sorted0);
  s.sorted[1] = (uint2*)(ws + l.sorted1);
  const size_t smem = ((size_t)(kSortWarps + 2) << s.digit_bits) * 4;
  DASH_TRY(allow_shared((const void*)embed_sort_kernel, (int)(((size_t)(kSortWarps + 2) << kMaxDigitBits) * 4)));
  embed_sort_kernel<<<kSortCtas, kSortThreads, smem, stream>>>(s);
  DASH_TRY(cudaGetLastError());
  if (!accumulate)
    DASH_TRY(launch_after(embed_zero_kernel, dim3((unsigned)zero_blocks), kZeroThreads, 0, stream, (char*)dtable,
                          table_bytes));
  RowArgs a;
  a.sorted = s.sorted[(s.passes - 1) & 1];
  a.T = T;
  a.V = V;
  a.D = D;
  a.ld_dout = ld_dout;
  a.scale = scale;
  a.accumulate = accumulate;
  a.part = (float*)(ws + l.part);
  a.Dp = l.Dp;
  a.runs = l.runs;
  if (dout_dtype == DASH_BF16)
    return dtable_dtype == DASH_BF16 ? rows_typed<__nv_bfloat16, __nv_bfloat16>(dout, dtable, a, stream)
                                     : rows_typed<__nv_bfloat16, float>(dout, dtable, a, stream);
  if (dout_dtype == DASH_FP16)
    return dtable_dtype == DASH_FP16 ? rows_typed<__half, __half>(dout, dtable, a, stream)
                                     : rows_typed<__half, float>(dout, dtable, a, stream);
  return rows_typed<float, float>(dout, dtable, a, stream);
}

}  // extern "C"
