// Softmax cross entropy from hidden states (X [T, D], W [V, D], both bf16) without stored
// logits, and its gradient. Four products share one persistent tensor-core kernel's code:
//   LSE   Z = X W^T        a 256 x 256 tile of logits is reduced to (max, sum of exp2) per
//                          row and half tile; the target's logit is stored
//   GRAD  Z = X W^T again  the tile becomes G = g (exp(z - lse) - [v = y]) in bf16
//   DX    dX = G W         K = the vocabulary (of one piece), W read N-major
//   DW    dW = G^T X       K = the tokens, both operands MN-major
// G is rounded no more than the results: it is one bf16 term where they are bf16. Up to 128 tokens
// half of a tile's rows would be empty: there G is held as two terms, the second one what the
// first one's rounding left; DX puts the second terms into the other half (its join adds them),
// DW takes them as 128 more tokens, and neither takes longer. An fp32 dW of more tokens gets the
// two terms too, as twice as many tokens (DX, which is bf16, the first alone).
// DX and DW of a piece share a launch (BOTH) where they are few tiles (kTogetherRounds): neither
// reads what the other writes, and their tiles fill the chip's last round together.
// A unit of work is one output tile of 256 x 256 (for DX one K range of it), dealt round robin
// to pairs of CTAs on neighbouring SMs (cta_group::2): each CTA loads its 128 rows of A and
// its 128 columns of B, one thread of the pair issues MMAs of 256 x 256 x 16 over both, and
// each CTA's TMEM gets its 128 rows of the product. So an SM reads half of B that a tile of
// its own would need.
//
// Bound by the tensor cores, over a whole pass by the power they draw. Measured at 8192 tokens,
// 65536 ids, D = 4096: LSE 2.35 ms, GRAD, DX and DW of a quarter of the ids 0.59, 0.60 and 0.61
// ms by themselves (1800 to 1870 TFLOP/s), the four in a loop 10.5 ms (1675; cuBLAS sustains
// 1683 on this card), 10.95 on another. With an fp32 dW the backward takes 11.1 ms instead of 7.8. Tiles of 128 x 256 on single CTAs: 0.65 to 0.67 ms, 11.5 ms in a loop.
//
// Warp roles (384 threads a CTA): 0 = TMA producer (64 of K per stage, 6 stages of 32 KB), 1 =
// MMA issuer (the pair's first CTA), 4..11 = epilogue (one 32-row quarter and one half of the
// columns each). Two 256-column accumulators in TMEM, so that the next tile's MMAs run while
// one is read out.
//
// Barriers: a stage's FULL and an accumulator's EMPTY live in the first CTA, where the issuer
// waits for both CTAs' copies and read-outs; a stage's EMPTY and an accumulator's FULL live in
// both, arrived at by the issuer's commits.
#pragma once

#include "tc_shared.cuh"
#include "train_common.cuh"

namespace dash {
namespace xent {

using namespace dash::tc;

enum Op : int { LSE = 0, GRAD = 1, DX = 2, DW = 3, BOTH = 4 };

// What DX does with a finished tile, and DW by type and accumulation.
enum OutMode : int {
  OUT_BF16 = 0,        // dX or dW, final
  OUT_F32 = 1,         // dW in fp32, final; dX of the first of several pieces
  OUT_F32_ADD = 2,     // dX += (a middle piece); dW fp32 accumulated
  OUT_BF16_ADD = 3,    // dX final = fp32 sum of the pieces before + this one; dW bf16 accumulated
  OUT_PART = 4         // dX: this K range's partial
};

struct Params {
  int M, N, K;               // extents of this product (valid rows, columns, K)
  int b_row0;                // LSE/GRAD/DX: first vocabulary row of the piece
  int tiles_m, tiles_n, splits, ksteps_per_split;
  int id_bits;
  const void* targets;
  long long ignore_index;
  float scale, scale_log2;
  // LSE
  float2* part;              // [2 * tiles_n][M]
  float* ztgt;               // [M]
  // GRAD
  const float* lse;
  const float* dloss;
  __nv_bfloat16* g;          // [M][ldg]
  __nv_bfloat16* g2;         // G's second terms, laid out as g, or null
  long long ldg;
  long long V;
  // DX, DW
  int out_mode;
  void* out;                 // dx, or dw at the piece's first row
  float* acc;                // DX: fp32 [M][N] over the pieces, or the K ranges' partials
  int* header;
  long long timeout_ns;
  int seg_steps;             // DX, DW: K steps of a segment
  int two;                   // DX: the second terms lie in the tile's other half
  int rows;                  // tokens
  int withhold;              // testing hook: load no tiles, so the waits for them run out
};

struct Maps {
  CUtensorMap a, b;
  CUtensorMap a2;            // DX, DW: G's second terms
  CUtensorMap c;             // DW, not accumulated: the output, boxes of 32 rows x 128 bytes
};
constexpr int kTwoTermRows = 128;

constexpr int kXentThreads = 384;
constexpr int kTM = 256, kTN = 256, kTK = 64;         // of a pair
constexpr int kCtaM = kTM / 2, kCtaN = kTN / 2;       // what one CTA loads
constexpr int kStages = 6;
constexpr int kGroupM = 8;
constexpr int kABytes = kCtaM * kTK * 2, kBBytes = kCtaN * kTK * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kBarOff = kStages * kStageBytes;
// DW stores its tiles from shared memory, 32 rows x 128 bytes a warp at a time: whole lines. For
// few tokens its stores are all there is: gradients of 128 tokens x 65536 ids x 2048 take 201 us,
// 215 with 32 bytes of a row a thread.
constexpr int kStoreOff = kBarOff + 1024, kStoreBytes = 4096;
// DX and DW run in one launch up to this many units a pair of SMs. Backward pass, two launches /
// one: 333 tokens x 5003 ids at D = 64, 1024, 4096 (1, 2, 5 a pair) 19.8 / 15.3, 33.4 / 28.8,
// 64.0 / 59.7 us; 64 x 32768 at 1024 (7.7) 61.7 / 60.2; 1024 x 32768 at 1024 (7.6) 143.3 / 143.3;
// 2048 x 32768 at 2048 (14) 504.3 / 505.4; 128 x 65536 at 2048 (28) 203 / 210, where reads of W
// then run among writes of dW.
constexpr int kTogetherRounds = 8;

template <int OP>
constexpr int kSmem = (OP == DW || OP == BOTH ? kStoreOff + 8 * kStoreBytes : kBarOff + 256) + 1024;
static_assert(kSmem<BOTH> <= 232448, "shared memory budget");
// LSE sums K in segments of 1024: the tensor core truncates its fp32 additions, which over
// 4096 of K made lse 1.7e-5 too small (2.2e-6 of it; fp32 multiply-adds to nearest: 3.9e-7); a
// segment's sum is added in registers, to nearest, while the next one is computed. Segments of
// 512, 1024, 2048: errors of 2.6e-7, 5.4e-7, 1.1e-6, and 1.9, 0.7, 0.2 % more time for the step
// above. GRAD needs none: its logits go into G, which is rounded more. DX and DW sum long axes,
// where truncation is a bias that grows with K: terms of one sign lose some 2^-25.5 of their sum
// with each 16 of K (dW of 262144 such tokens was 3e-4 too small). bf16 results get segments of
// 16384 ids or tokens, which leave 2^-15.5, an fp32 dW segments of 4096 tokens, 2^-17.5 and less
// than G's rounding. Kernels for K of one segment are compiled without (SEGMENTS), which spares
// the backward of 8192 tokens 3 %.
constexpr int kSegSteps = 1024 / kTK;
constexpr int kSegSteps16 = 16384 / kTK, kSegSteps32 = 4096 / kTK;
template <int OP, bool SEGMENTS>
__device__ __forceinline__ int seg_steps(const Params& p) {
  return OP == LSE ? kSegSteps : SEGMENTS ? p.seg_steps : 1 << 30;
}
enum { B_FULL = 0, B_EMPTY = B_FULL + kStages, B_ACC_FULL = B_EMPTY + kStages,
       B_ACC_EMPTY = B_ACC_FULL + 2, B_DRAIN = B_ACC_EMPTY + 2, B_COUNT };
static_assert(8 * B_COUNT + 8 <= 256, "barrier space");

// Unit -> (m tile, n tile, K range). Tiles are numbered in groups of kGroupM m-tiles, m
// first, so that concurrent units share their A and B panels in L2.
__device__ __forceinline__ void unit_of(const Params& p, int u, int& mi, int& ni, int& split) {
  split = u % p.splits;
  const int tile = u / p.splits;
  const int per_group = kGroupM * p.tiles_n;
  const int first_m = (tile / per_group) * kGroupM;
  const int gm = min(kGroupM, p.tiles_m - first_m);
  const int r = tile % per_group;
  mi = first_m + r % gm;
  ni = r / gm;
}

// 32 bytes of one output row in one store (`wide`: the address is a multiple of 32) or two: a
// thread owns a row, so its store should fill a whole 32-byte sector of L2 (16-byte stores wrote
// each sector up to three times: gradients of 128 tokens x 65536 ids x 2048 took 240 us, 203 so).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 32 consecutive columns of one output row: fp32 values to bf16 or fp32, added to what is
// there (or in `old32`) where the mode says so. `n` columns are valid (a multiple of 8).
template <bool ADD>
__device__ __forceinline__ void put_bf16(__nv_bfloat16* dst, const float* old32, const float (&v)[32],
                                         int n, bool wide) {
#pragma unroll
  for (int c = 0; c < 32; c += 16) {
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[c + h + i];
      if (ADD && c + h < n) {
        float o[8];
        if (old32) train::load_f32<float, 8>(old32 + c + h, o);
        else train::load_f32<__nv_bfloat16, 8>(dst + c + h, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += o[i];
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) w[(h + i) >> 1] = ptx::pack_bf16(x[i], x[i + 1]);
    }
    if (c + 8 < n) store32(dst + c, w, wide);
    else if (c < n) *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <bool ADD>
__device__ __forceinline__ void put_f32(float* dst, const float (&v)[32], int n, bool wide) {
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    if (c < n) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[c + i];
      if (ADD) {
        float o[8];
        train::load_f32<float, 8>(dst + c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += o[i];
      }
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
      store32(dst + c, w, wide);
    }
  }
}

// A warp's 32 rows x 128 columns of dW from its accumulator, through its place in shared memory
// (rows of 128 bytes, 16-byte chunks swizzled as the tensor map has them).
template <bool F32>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint8_t* buf, uint32_t tmem_from, int col,
                                           int row0, int rows, int cols, int lane) {
  constexpr int W = F32 ? 32 : 64;                         // columns of 128 bytes
#pragma unroll 1
  for (int c0 = 0; c0 < kTN / 2; c0 += W) {
    if (lane == 0) ptx::bulk_wait_read_all();              // the last store has left the buffer
    __syncwarp();
#pragma unroll
    for (int q = 0; q < W; q += 32) {
      float v[32];
      ptx::tmem_ld32(tmem_from + c0 + q, v);
      constexpr int CH = F32 ? 8 : 4;                      // 16-byte chunks of 32 columns
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (q / 32) * CH + i;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = F32 ? __float_as_uint(v[4 * i + k]) : ptx::pack_bf16(v[(8 * i + 2 * k) & 31], v[(8 * i + 2 * k + 1) & 31]);
        ptx::st_shared_v4(ptx::smem_u32(buf) + lane * 128 + ((c ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < rows && col + c0 < cols) {
      ptx::tma_store_2d(map, buf, col + c0, row0);
      ptx::bulk_commit();
    }
  }
}

// What the roles of a CTA share.
struct Cta {
  uint8_t* sm;
  uint64_t* bars;
  volatile int* abort_flag;
  uint32_t tmem;
  int rank, warp, lane;        // rank 0: the pair's first CTA
  long long tmo;
};
template <int OP>
constexpr bool kAMn = OP == DW;
template <int OP>
constexpr bool kBMn = OP == DX || OP == DW;
// K steps of one of G's terms, and of a unit's whole K.
__device__ __forceinline__ int ksteps_one(const Params& p) { return (p.K + kTK - 1) / kTK; }
template <int OP>
__device__ __forceinline__ int ksteps_all(const Params& p) {
  return OP == DW && p.g2 ? 2 * ksteps_one(p) : ksteps_one(p);
}
__device__ __forceinline__ int units_of(const Params& p) { return p.tiles_m * p.tiles_n * p.splits; }

// TMA producer, one unit. kb: K blocks so far.
template <int OP>
__device__ __forceinline__ void load_unit(const Params& p, const Maps& maps, const Cta& c, int u, long long& kb,
                                          bool& ok) {
  constexpr bool A_MN = kAMn<OP>, B_MN = kBMn<OP>;
  uint8_t* sm = c.sm;
  uint64_t* bars = c.bars;
  volatile int* abort_flag = c.abort_flag;
  const int rank = c.rank, ksteps1 = ksteps_one(p), ksteps = ksteps_all<OP>(p);
  const long long tmo = c.tmo;
  int mi, ni, split;
  unit_of(p, u, mi, ni, split);
  const int m0 = mi * kTM + rank * kCtaM, n0 = ni * kTN + rank * kCtaN;
  const int k_end = min(ksteps, (split + 1) * p.ksteps_per_split);
  for (int k = split * p.ksteps_per_split; k < k_end; ++k, ++kb) {
    const int s = (int)(kb % kStages);
    if (kb >= kStages &&
        !(ok = ptx::mbar_wait(bars + B_EMPTY + s, (int)((kb / kStages) - 1) & 1, abort_flag, tmo)))
      break;
    // the first CTA expects both CTAs' bytes; the other's may arrive before that
    const uint32_t full = ptx::peer_smem(bars + B_FULL + s, 0);
    if (rank == 0) ptx::mbar_expect_tx(bars + B_FULL + s, 2 * kStageBytes);
    uint8_t* sa = sm + s * kStageBytes;
    uint8_t* sb = sa + kABytes;
    int row = m0;
    const bool second = OP == DW && k >= ksteps1;
    const int k0 = (second ? k - ksteps1 : k) * kTK;
    const CUtensorMap* map_a = second ? &maps.a2 : &maps.a;
    if (OP == DX && p.two && rank == 1) {
      map_a = &maps.a2;
      row = 0;
    }
    if (A_MN) {
      for (int i = 0; i < kCtaM / 64; ++i)
        ptx::tma_load_2d_pair(sa + i * 8192, map_a, row + i * 64, k0, full);
    } else {
      ptx::tma_load_2d_pair(sa, map_a, k0, row, full);
    }
    if (B_MN) {
      const int kr = OP == DX ? p.b_row0 + k0 : k0;
      for (int i = 0; i < kCtaN / 64; ++i)
        ptx::tma_load_2d_pair(sb + i * 8192, &maps.b, n0 + i * 64, kr, full);
    } else {
      ptx::tma_load_2d_pair(sb, &maps.b, k0, p.b_row0 + n0, full);
    }
  }
}

// MMA issuer, one unit (one thread of the pair's first CTA). it: accumulators filled so far.
template <int OP, bool SEGMENTS>
__device__ __forceinline__ void issue_unit(const Params& p, const Cta& c, int u, long long& kb, int& it,
                                           bool& ok) {
  constexpr bool A_MN = kAMn<OP>, B_MN = kBMn<OP>;
  constexpr uint32_t ID = ptx::idesc_bf16(kTM, kTN, A_MN, B_MN);
  // a K step of 16: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major block
  constexpr uint32_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;
  uint64_t* bars = c.bars;
  volatile int* abort_flag = c.abort_flag;
  const uint32_t s0 = ptx::smem_u32(c.sm), tmem = c.tmem;
  const int ksteps = ksteps_all<OP>(p);
  const long long tmo = c.tmo;
  int mi, ni, split;
  unit_of(p, u, mi, ni, split);
  const int u_end = min(ksteps, (split + 1) * p.ksteps_per_split), seg = seg_steps<OP, SEGMENTS>(p);
  for (int k_begin = split * p.ksteps_per_split; k_begin < u_end; k_begin += seg, ++it) {
    const int acc = it & 1;
    const int k_end = OP == LSE || SEGMENTS ? min(u_end, k_begin + seg) : u_end;
    if (it >= 2 && !(ok = ptx::mbar_wait(bars + B_ACC_EMPTY + acc, ((it >> 1) - 1) & 1, abort_flag, tmo)))
      break;
    ptx::tc_fence_after();
    for (int k = k_begin; k < k_end; ++k, ++kb) {
      const int s = (int)(kb % kStages);
      if (!(ok = ptx::mbar_wait(bars + B_FULL + s, (int)(kb / kStages) & 1, abort_flag, tmo))) break;
      ptx::tc_fence_after();
      const uint32_t a_lo = ptx::sdesc_lo(s0 + s * kStageBytes, A_MN ? 8192 : 16);
      const uint32_t b_lo = ptx::sdesc_lo(s0 + s * kStageBytes + kABytes, B_MN ? 8192 : 16);
#pragma unroll
      for (int ks = 0; ks < kTK / 16; ++ks)
        ptx::mma_lo_pair(tmem + acc * kTN, a_lo + ks * A_STEP, b_lo + ks * B_STEP, ID,
                         (k > k_begin || ks > 0) ? 1u : 0u);
      ptx::mma_commit_pair(bars + B_EMPTY + s);
    }
    if (!ok) break;
    ptx::mma_commit_pair(bars + B_ACC_FULL + acc);
  }
}

// Adds the next accumulator's part of a thread's row to z, or sets z to it at the first one.
__device__ __forceinline__ void add_segment(float (&z)[kTN / 64][32], uint32_t from, bool first) {
#pragma unroll
  for (int c = 0; c < kTN / 64; ++c) {
    if (first) {
      ptx::tmem_ld32(from + c * 32, z[c]);
    } else {
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        float t[16];
        ptx::tmem_ld16(from + c * 32 + h, t);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[c][h + i] += t[i];
      }
    }
  }
}

// Epilogue, one unit: a warp's 32 rows and half of the columns.
template <int OP, bool SEGMENTS>
__device__ __forceinline__ void finish_unit(const Params& p, const Maps& maps, const Cta& c, int u, int& it,
                                            bool& ok) {
  uint8_t* sm = c.sm;
  uint64_t* bars = c.bars;
  volatile int* abort_flag = c.abort_flag;
  const int rank = c.rank, warp = c.warp, lane = c.lane, ksteps = ksteps_all<OP>(p);
  const uint32_t tmem = c.tmem;
  const long long tmo = c.tmo;
  const int quarter = warp & 3, half = (warp - 4) >> 2;
  const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
  int mi, ni, split;
  unit_of(p, u, mi, ni, split);
  const int row = mi * kTM + rank * kCtaM + quarter * 32 + lane;
  const int col0 = ni * kTN + half * (kTN / 2);
  const bool live = OP == DX && p.two ? (row & (kTwoTermRows - 1)) < p.rows : row < p.M;
  // what the row needs besides the tile, fetched before the wait
  long long tgt = -1;
  float nlse2 = 0.f, gs = 0.f;
  if (OP == LSE || OP == GRAD) {
    if (live) tgt = train::load_index(p.targets, row, p.id_bits);
    if (OP == GRAD && live) {
      const bool used = tgt != p.ignore_index && tgt >= 0 && tgt < p.V;
      gs = used ? p.scale * __ldg(p.dloss + row) : 0.f;
      nlse2 = -__ldg(p.lse + row) * kLog2e;
      if (!used) tgt = -1;
    }
    if (tgt == p.ignore_index) tgt = -1;
    tgt -= p.b_row0;
  }
  if constexpr (OP == LSE) {
    float z[kTN / 64][32];
    for (int k = 0; k < ksteps; k += kSegSteps, ++it) {
      const int acc = it & 1;
      if (!(ok = ptx::warp_wait(bars + B_ACC_FULL + acc, (it >> 1) & 1, abort_flag, tmo))) break;
      ptx::tc_fence_after();
      const uint32_t from = tmem + lane_addr + acc * kTN + half * (kTN / 2);
      add_segment(z, from, k == 0);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_peer(ptx::peer_smem(bars + B_ACC_EMPTY + acc, 0));
    }
    if (!ok) return;
    float m2 = -INFINITY, sum = 0.f;
#pragma unroll
    for (int c0 = 0; c0 < kTN / 2; c0 += 32) {
      float (&v)[32] = z[c0 / 32];
      const int col = col0 + c0;                       // first column of the 32
      const int n = p.N - col;                         // valid ones
      if (n > 0) {
        const long long tc = tgt - col;
        float cm = -INFINITY;
        float zt = 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (c == tc) zt = v[c];
          v[c] = c < n ? v[c] * p.scale_log2 : -INFINITY;
          cm = fmaxf(cm, v[c]);
        }
        if (tc >= 0 && tc < 32 && tc < n) p.ztgt[row] = zt * p.scale;
        const float nm = fmaxf(m2, cm);
        const float base = nm == -INFINITY ? 0.f : nm;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) s += ptx::ex2(v[c] - base);
        sum = sum * ptx::ex2(m2 - base) + s;
        m2 = nm;
      }
    }
    if (live) p.part[(size_t)(ni * 2 + half) * p.M + row] = make_float2(m2, sum);
    return;
  }
  if constexpr (SEGMENTS) {
    // all segments but the last into registers, and their sum to the last one's place in TMEM
    const int k0 = split * p.ksteps_per_split, n = min(ksteps, k0 + p.ksteps_per_split) - k0;
    if (n > p.seg_steps) {
      float z[kTN / 64][32];
#pragma unroll 1
      for (int k = 0;;) {
        const int acc = it & 1;
        if (!(ok = ptx::warp_wait(bars + B_ACC_FULL + acc, (it >> 1) & 1, abort_flag, tmo))) return;
        ptx::tc_fence_after();
        const uint32_t from = tmem + lane_addr + acc * kTN + half * (kTN / 2);
        add_segment(z, from, k == 0);
        k += p.seg_steps;
        if (k >= n) {
#pragma unroll
          for (int c = 0; c < kTN / 64; ++c)
            ptx::tmem_st32(from + c * 32, reinterpret_cast<const uint32_t(&)[32]>(z[c]));
          break;
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_peer(ptx::peer_smem(bars + B_ACC_EMPTY + acc, 0));
        ++it;
      }
    }
  }
  const int acc = it & 1;
  if (!(ok = ptx::warp_wait(bars + B_ACC_FULL + acc, (it >> 1) & 1, abort_flag, tmo))) return;
  ptx::tc_fence_after();
  const uint32_t from = tmem + lane_addr + acc * kTN + half * (kTN / 2);
  const bool by_tile = OP == DW && (p.out_mode == OUT_BF16 || p.out_mode == OUT_F32);
  if (OP == DW && by_tile) {
    uint8_t* buf = sm + kStoreOff + (warp - 4) * kStoreBytes;
    const int row0 = row - lane;
    if (p.out_mode == OUT_F32) store_tile<true>(&maps.c, buf, from, col0, row0, p.M, p.N, lane);
    else store_tile<false>(&maps.c, buf, from, col0, row0, p.M, p.N, lane);
  }
#pragma unroll 1
  for (int c0 = 0; c0 < (by_tile ? 0 : kTN / 2); c0 += 32) {
    float v[32];
    ptx::tmem_ld32(from + c0, v);
    const int col = col0 + c0;                       // first column of the 32
    const int n = p.N - col;                         // valid ones
    if (OP == GRAD) {
      const long long tc = tgt - col;
      uint32_t w[16], w2[16];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float a = ptx::ex2(fmaf(v[c], p.scale_log2, nlse2));
        float b = ptx::ex2(fmaf(v[c + 1], p.scale_log2, nlse2));
        if (c == tc) a -= 1.f;
        if (c + 1 == tc) b -= 1.f;
        a = gs == 0.f ? 0.f : a * gs;
        b = gs == 0.f ? 0.f : b * gs;
        w[c >> 1] = ptx::pack_bf16(a, b);
        if (p.g2)
          w2[c >> 1] = ptx::pack_bf16(a - __uint_as_float(w[c >> 1] << 16),
                                      b - __uint_as_float(w[c >> 1] & 0xffff0000u));
      }
      if (live && n > 0) {
        __nv_bfloat16* dst = p.g + (size_t)row * p.ldg + col;     // ldg: a multiple of 256
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t h[8] = {w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                 w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
          store32(dst + 16 * i, h, true);
          if (p.g2) {
            const uint32_t l[8] = {w2[8 * i], w2[8 * i + 1], w2[8 * i + 2], w2[8 * i + 3],
                                   w2[8 * i + 4], w2[8 * i + 5], w2[8 * i + 6], w2[8 * i + 7]};
            store32(p.g2 + (size_t)row * p.ldg + col + 16 * i, l, true);
          }
        }
      }
    } else {
      if (live && n > 0) {
        const size_t at = (size_t)row * p.N + col;
        __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(p.out) + at;
        float* of = (OP == DX ? p.acc + (p.out_mode == OUT_PART ? (size_t)split * p.M * p.N : 0)
                              : reinterpret_cast<float*>(p.out)) + at;
        const bool wide16 = ((uintptr_t)ob & 31) == 0, wide32 = ((uintptr_t)of & 31) == 0;
        if (p.out_mode == OUT_BF16) put_bf16<false>(ob, nullptr, v, n, wide16);
        else if (p.out_mode == OUT_BF16_ADD) put_bf16<true>(ob, OP == DX ? of : nullptr, v, n, wide16);
        else if (p.out_mode == OUT_F32_ADD) put_f32<true>(of, v, n, wide32);
        else put_f32<false>(of, v, n, wide32);
      }
    }
  }
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive_peer(ptx::peer_smem(bars + B_ACC_EMPTY + acc, 0));
  ++it;
}

// The second product of a launch: DW's in BOTH, else nothing.
template <int OP>
struct Second {};
template <>
struct Second<BOTH> {
  Params p;
  Maps maps;
};

template <int OP, bool SEGMENTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXentThreads, 1)
    gemm_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps,
                const __grid_constant__ Second<OP> second) {
  constexpr int OP1 = OP == BOTH ? DX : OP;
  extern __shared__ uint8_t smem_xent[];
  train::grid_next();
  Cta c;
  c.sm = (uint8_t*)(((uintptr_t)smem_xent + 1023) & ~(uintptr_t)1023);
  c.bars = (uint64_t*)(c.sm + kBarOff);
  uint32_t* tmem_slot = (uint32_t*)(c.sm + kBarOff + 8 * B_COUNT);
  c.abort_flag = (volatile int*)(c.sm + kBarOff + 8 * B_COUNT + 4);
  c.warp = threadIdx.x >> 5;
  c.lane = threadIdx.x & 31;
  c.rank = (int)ptx::cluster_rank();
  c.tmo = p.timeout_ns;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units1 = units_of(p);
  int units = units1;
  if constexpr (OP == BOTH) units += units_of(second.p);

  if (threadIdx.x == 0) {
    ptx::prefetch_map(&maps.a);
    ptx::prefetch_map(&maps.b);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(c.bars + B_FULL + s, 1);
      ptx::mbar_init(c.bars + B_EMPTY + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(c.bars + B_ACC_FULL + a, 1);
      ptx::mbar_init(c.bars + B_ACC_EMPTY + a, 16);        // 8 epilogue warps of each CTA
    }
    ptx::mbar_init(c.bars + B_DRAIN, 1);
    *c.abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncwarp();
  if (c.warp == 1) ptx::tmem_alloc_pair(tmem_slot, 512);
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  c.tmem = *tmem_slot;
  train::grid_wait();

  long long kb = 0;
  int it = 0;
  bool ok = true;
  if (c.warp == 0) {
    if (c.lane == 0) {
      ok = p.withhold == 0;
      for (int u = pair; ok && u < units; u += pairs) {
        if constexpr (OP == BOTH) {
          if (u >= units1) {
            load_unit<DW>(second.p, second.maps, c, u - units1, kb, ok);
            continue;
          }
        }
        load_unit<OP1>(p, maps, c, u, kb, ok);
      }
    }
  } else if (c.warp == 1) {
    if (c.lane == 0 && c.rank == 0) {
      for (int u = pair; ok && u < units; u += pairs) {
        if constexpr (OP == BOTH) {
          if (u >= units1) {
            issue_unit<DW, false>(second.p, c, u - units1, kb, it, ok);
            continue;
          }
        }
        issue_unit<OP1, SEGMENTS>(p, c, u, kb, it, ok);
      }
      ptx::mma_commit_pair(c.bars + B_DRAIN);
    }
  } else if (c.warp >= 4) {
    for (int u = pair; ok && u < units; u += pairs) {
      if constexpr (OP == BOTH) {
        if (u >= units1) {
          finish_unit<DW, false>(second.p, second.maps, c, u - units1, it, ok);
          continue;
        }
      }
      finish_unit<OP1, SEGMENTS>(p, maps, c, u, it, ok);
    }
    if ((OP == DW || OP == BOTH) && c.lane == 0) ptx::bulk_wait_all();   // the stores have been performed
  }

  // Every MMA and with it every copy of the pair has ended once DRAIN completes; neither CTA
  // leaves before the other, whose barriers and copies it may signal.
  if (threadIdx.x == 0) ptx::mbar_drain(c.bars + B_DRAIN, 0, 1000000000ll);
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (c.warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(c.tmem, 512);
  }
  if (threadIdx.x == 0 && *c.abort_flag && atomicCAS(p.header + WS_STATUS, 0, kStatusSyncTimeout) == 0) {
    p.header[WS_BH] = -1;
    p.header[WS_QTILE] = blockIdx.x;
  }
}

__device__ __forceinline__ void add_part(float& m, float& s, const float2& x) {
  const float nm = fmaxf(m, x.x);
  const float base = nm == -INFINITY ? 0.f : nm;
  s = s * ptx::ex2(m - base) + x.y * ptx::ex2(x.x - base);
  m = nm;
}

// Joins the half tiles' (max, sum) of every row in a fixed order: 32 rows a block, the parts
// cut into 32 runs, a warp each, 8 loads in flight; then the runs in order.
__global__ void __launch_bounds__(1024) lse_join_kernel(const float2* part, const float* ztgt, int parts,
                                                        int T, const void* targets, int id_bits,
                                                        long long ignore_index, long long V, float* loss,
                                                        float* lse, int* header) {
  __shared__ float2 runs[32][32];
  train::grid_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f;
  if (row < T) {
    const int per = (parts + 31) / 32;
    const int end = min(parts, (g + 1) * per);
    int k = g * per;
    for (; k + 8 <= end; k += 8) {
      float2 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = part[(size_t)(k + i) * T + row];
#pragma unroll
      for (int i = 0; i < 8; ++i) add_part(m, s, x[i]);
    }
    for (; k < end; ++k) add_part(m, s, part[(size_t)k * T + row]);
  }
  runs[g][lane] = make_float2(m, s);
  __syncthreads();
  if (g == 0 && row < T) {
    for (int k = 1; k < 32; ++k) add_part(m, s, runs[k][lane]);
    const float l = (m == -INFINITY ? 0.f : m) * kLn2 + logf(s);
    lse[row] = l;
    const long long y = train::load_index(targets, row, id_bits);
    float out = 0.f;
    if (y != ignore_index) {
      if (y < 0 || y >= V) {
        train::report_index(header, CHK_TARGET, row, y, V);
        out = NAN;
      } else {
        out = l - ztgt[row];
      }
    }
    loss[row] = out;
  }
}

// dX from the K ranges' partials of n values each, added in order (after what the pieces before
// left in acc, when there are any), each with its second term's `second` values on where there
// is one; the last piece stores bf16. 4 columns a thread, 8 loads in flight.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) dx_join_kernel(const float* part, int splits, size_t n,
                                                               size_t stride, size_t second, float* acc,
                                                               int first, int last, __nv_bfloat16* dx) {
  const size_t i = ((size_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  train::grid_next();
  train::grid_wait();
  if (i >= n) return;
  float x[4] = {};
  if (!first) train::load_f32<float, 4>(acc + i, x);
  auto add = [&](const train::Vec<float, 4>& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] += __uint_as_float(v.w[k]);
  };
  for (int term = 0; term < (second ? 2 : 1); ++term) {
    const float* from = part + term * second + i;
    int s = 0;
    for (; s + 8 <= splits; s += 8) {
      train::Vec<float, 4> v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = train::load_vec<float, 4>(from + (s + k) * stride);
#pragma unroll
      for (int k = 0; k < 8; ++k) add(v[k]);
    }
    for (; s < splits; ++s) add(train::load_vec<float, 4>(from + s * stride));
  }
  if (last) {
    *reinterpret_cast<uint2*>(dx + i) = make_uint2(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]));
  } else {
    train::store_f32<float, 4>(acc + i, x);
  }
}

// Clears the header and reports targets out of range (the backward treats them as ignored).
__global__ void __launch_bounds__(1024) check_targets_kernel(const void* targets, int id_bits, int T,
                                                             long long ignore_index, long long V,
                                                             int* header) {
  train::grid_next();
  if (threadIdx.x < kWsHeaderBytes / 4) header[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 4
  for (unsigned t = threadIdx.x; t < (unsigned)T; t += 1024) {     // T may be within 1024 of 2^31
    const long long y = train::load_index(targets, t, id_bits);
    if (y != ignore_index && (y < 0 || y >= V)) train::report_index(header, CHK_TARGET, t, y, V);
  }
}

}  // namespace xent
}  // namespace dash
