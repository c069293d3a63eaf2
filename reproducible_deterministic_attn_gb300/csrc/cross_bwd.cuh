// Cross attention backward: dV = P^T dO, dS = P * (dO V^T - Delta), dQ = scale dS K,
// dK = scale dS^T Q with P = exp(scale Q K^T - LSE) recomputed and Delta = rowsum(dO * O).
//
// A unit of work is a segment of a group's row tiles against a segment of its key tiles; one CTA
// (of a persistent grid) takes the unit's key tiles one after the other, each against all the
// unit's row tiles. A task is one 128 x 128 tile of scores, with the keys in the TMEM lanes:
//   S^T   = K Q^T              M = 128 keys, N = 128 rows, K = D          TMEM cols [0, 128)
//   P^T   = exp2(S^T scale log2e - LSE log2e)            bf16, TMEM, over S^T's columns
//   dP^T  = V dO^T             M = 128 keys, N = 128 rows, K = D          TMEM cols [128, 256)
//   dS^T  = P^T * (dP^T - Delta)                         bf16, TMEM over S^T, and smem [key][row]
//   dV   += P^T dO             M = 128 keys, N = D, K = 128 rows, A from TMEM  [256, +DT)
//   dK   += dS^T Q             M = 128 keys, N = D, K = 128 rows, A from TMEM  [256 + DT, +DT)
//   dQ^T  = K^T dS^T           M = 128 (d), N = 128 rows, K = keys        TMEM cols [128, 256)
// dK and dV stay in TMEM over the unit's row tiles. dQ^T leaves TMEM with every task: of a single
// key tile it is the result (rounded to bf16 at once), else it is added over the unit's key tiles
// in fp32 in global memory (which L2 holds), always by the same thread: stored by the first key
// tile, added by the next ones, read back, added and rounded by the last.
// So no CTA waits for another one. Units that share key tiles leave fp32 partials of dK and dV,
// units that share row tiles partials of dQ; cross_grad_join_kernel adds them in order.
//
// Delta and -LSE log2e come per row from cross_pre_kernel, with -inf for rows a tile does not
// have (P = 0 there). Keys that a length leaves out: warp 2 zeroes their rows of K and V in shared
// memory, as they may hold anything, and their P is set to 0.
//
// Warp roles (512 threads): 0 = TMA producer, 1 = MMA issuer, 2 = key rows behind a length, 3 idle,
// 4..11 = softmax gradient (quarter = TMEM lanes = keys, half = 64 rows each), 12..15 = dQ
// read-out and the epilogue of dK and dV. Every wait is bounded.
#pragma once

#include "bwd_main.cuh"
#include "cross_common.cuh"

namespace dash {
namespace cross {

struct BwdArgs {
  Shape s;
  float* nnl;                // [group][tile][128] -LSE log2e
  float* delta;              // [group][tile][128]
  const __nv_bfloat16 *o, *dO;
  const float* lse;
  __nv_bfloat16 *dq, *dk, *dv;
  long long dq_b, dq_s, dq_h, dk_b, dk_s, dk_h, dv_b, dv_s, dv_h;
  float* dq_acc;             // [key segment][group][tile][32][DT][4]: rows in fours, of each column
  float* dkv_part;           // [row segment][group][key tile][dK, dV][128][DT]
  int qsegs, qper, ksegs, kper;
  int units;
  float scale, scale_log2;
  int* header;
  long long timeout_ns;
  int withhold;
};

template <int DT>
struct BwdLay {
  static constexpr int TILE = kTile * DT * 2;
  static constexpr int DS_BYTES = kTile * kTile * 2;
  static constexpr int OFFS = 2 * kTile * 4;                   // -LSE log2e and Delta of a row tile
  static constexpr int NQ = DT == 64 ? 3 : 2;
  static constexpr int K_OFF = 0, V_OFF = TILE, Q_OFF = 2 * TILE;
  static constexpr int NDO = 2;
  static constexpr int DO_OFF = Q_OFF + NQ * TILE;
  static constexpr int DS_OFF = DO_OFF + NDO * TILE;
  // DT = 64: zeros after which K^T is padded to 128 rows, so that dQ^T is an M = 128 product
  static constexpr int ZERO_OFF = DS_OFF + DS_BYTES;
  static constexpr int ZERO_BYTES = DT == 64 ? TILE : 0;
  static constexpr int OFFS_OFF = ZERO_OFF + ZERO_BYTES;
  static constexpr int BAR_OFF = OFFS_OFF + NQ * OFFS;
  static constexpr int ALLOC = BAR_OFF + 256;                  // the base is 1024-aligned (checked)
  static_assert(ALLOC <= 232448, "shared memory budget");
  // DT = 64 leaves columns for dQ^T of its own; DT = 128 puts it where dP^T was
  static constexpr bool kSepDQ = DT == 64;
  static constexpr int T_SP = 0, T_DP = 128, T_DV = 256, T_DK = 256 + DT, T_DQ = kSepDQ ? 384 : T_DP;
  static constexpr int REGS_LAUNCH = 128, REGS_SINGLE = 88, REGS_READOUT = 168;
  static_assert(REGS_SINGLE + 2 * REGS_LAUNCH + REGS_READOUT == 4 * REGS_LAUNCH,
                "the four warpgroups must share exactly the launch's registers");
};

enum {
  C_KV_FULL = 0, C_KV_READY, C_KV_EMPTY, C_Q_FULL, C_Q_EMPTY = C_Q_FULL + 3, C_DO_FULL = C_Q_EMPTY + 3,
  C_DO_EMPTY = C_DO_FULL + 2, C_S_FULL = C_DO_EMPTY + 2, C_SP_FREE, C_P_FULL, C_DP_FULL, C_DS_FULL, C_DQ_FULL, C_DQ_EMPTY, C_ACC_FULL,
  C_ACC_EMPTY, C_DRAIN, C_COUNT
};
static_assert(8 * C_COUNT + 8 <= 256, "barrier area");

// A CTA's tasks: units u, u + grid, ..., of each the key tiles, of each the row tiles.
struct BwdWalk {
  const BwdArgs& p;
  int u, bh, b, hk, qseg, kseg, len;
  int q0, nqt, k0, nkt;      // the unit's first row tile and their number, its key tiles
  int i, j;                  // key tile, row tile within the unit
  __device__ __forceinline__ BwdWalk(const BwdArgs& a)
      : p(a), u((int)blockIdx.x - (int)gridDim.x), nqt(0), nkt(0), i(0), j(0) {}
  __device__ __forceinline__ bool next() {
    if (++j < nqt) return true;
    j = 0;
    if (++i < nkt) return true;
    i = 0;
    do {
      u += gridDim.x;
      if (u >= p.units) return false;
      kseg = u % p.ksegs;
      const int r = u / p.ksegs;
      qseg = r % p.qsegs;
      bh = r / p.qsegs;
      b = bh / p.s.Hk;
      hk = bh - b * p.s.Hk;
      len = length_of(p.s, b);
      q0 = qseg * p.qper;
      nqt = min(p.qper, p.s.ntile - q0);
      k0 = kseg * p.kper;
      nkt = max(0, min((max(len, 0) + kTile - 1) / kTile, k0 + p.kper) - k0);
    } while (nkt == 0);
    return true;
  }
  __device__ __forceinline__ int keys() const { return min(kTile, len - (k0 + i) * kTile); }
  __device__ __forceinline__ bool first_of_tile() const { return j == 0; }
  __device__ __forceinline__ bool last_of_tile() const { return j == nqt - 1; }
  __device__ __forceinline__ int tile() const { return q0 + j; }
};

// The K steps of a product of two K-major operands, of which `n` are taken.
template <int DT>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int n) {
#pragma unroll
  for (int ks = 0; ks < DT / 16; ++ks) {
    if (ks < n) ptx::mma_lo(d, a, b, id, ks > 0);
    a = ks == 3 ? next_k<3>(a) : next_k<0>(a);
    b = ks == 3 ? next_k<3>(b) : next_k<0>(b);
  }
}
// dQ^T's K steps K0 .. K1 - 1 of the n that hold keys (both operands MN-major).
template <int K0, int K1>
__device__ __forceinline__ void issue_dq(uint32_t d, uint32_t& a, uint32_t& b, uint32_t id, int n) {
#pragma unroll
  for (int ks = K0; ks < K1; ++ks) {
    if (ks < n) ptx::mma_lo(d, a, b, id, ks > 0);
    a = ptx::step_add<kMnStep>(a);
    b = ptx::step_add<kMnStep>(b);
  }
}

__device__ __forceinline__ void ld_relaxed_v4(const float* p, float* v) {
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "l"(p)
               : "memory");
}

// Delta = rowsum(dO * O) and -LSE log2e per row, in row tiles; 16 lanes a row. The first block
// clears the workspace's header and looks for lengths out of range.
__global__ void __launch_bounds__(256) cross_pre_kernel(const __grid_constant__ BwdArgs p) {
  train::grid_next();
  if (blockIdx.x == 0) {
    if (threadIdx.x < kWsHeaderBytes / 4) p.header[threadIdx.x] = 0;
    __syncthreads();
    if (p.s.lens)
      for (int b = threadIdx.x; b < p.s.B; b += blockDim.x)
        if (length_of(p.s, b) < 0)
          train::report_index(p.header, CHK_LENGTH, b, train::load_index(p.s.lens, b, p.s.id_bits), p.s.Sk);
  }
  const long long row = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  if (row >= (long long)p.s.B * p.s.Hk * p.s.ntile * kTile) return;      // whole halves of a warp
  const int r = (int)(row % kTile);
  const long long rest = row / kTile;
  const int tile = (int)(rest % p.s.ntile), bh = (int)(rest / p.s.ntile), b = bh / p.s.Hk, hk = bh - b * p.s.Hk;
  int token, head;
  const bool live = row_of(p.s, tile, r, token, head);
  const int h = hk * p.s.g + head;
  float t = 0.f;
  if (live && 8 * l < p.s.D) {
    const size_t at = (((size_t)b * p.s.Sq + token) * p.s.Hq + h) * p.s.D + 8 * l;
    float x[8], y[8];
    train::load_f32<__nv_bfloat16, 8>(p.o + at, x);
    train::load_f32<__nv_bfloat16, 8>(p.dO + at, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmaf(x[i], y[i], t);
  }
  const uint32_t half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(half, t, o);
  if (l == 0) {
    p.delta[row] = t;
    p.nnl[row] = live ? -kLog2e * p.lse[((size_t)b * p.s.Hq + h) * p.s.Sq + token] : -INFINITY;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    cross_bwd_kernel(const __grid_constant__ BwdArgs p, const __grid_constant__ Maps maps) {
  using L = BwdLay<DT>;
  extern __shared__ __align__(1024) uint8_t smem_crossb[];
  uint8_t* sm = smem_crossb;
  uint64_t* bars = (uint64_t*)(sm + L::BAR_OFF);
  uint32_t* tmem_slot = (uint32_t*)(sm + L::BAR_OFF + 8 * C_COUNT);
  volatile int* abort_flag = (volatile int*)(sm + L::BAR_OFF + 8 * C_COUNT + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long tmo = p.timeout_ns;
  const int dsteps = (p.s.D + 15) >> 4;

  train::grid_next();
  // The layout fills most of the opt-in maximum, so there is no room to realign the base.
  if (ptx::smem_u32(sm) & 1023u) {
    train::grid_wait();
    if (threadIdx.x == 0) atomicCAS(p.header + WS_STATUS, 0, kStatusSmemLayout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int k = 0; k < C_COUNT; ++k) {
      const int n = k == C_P_FULL || k == C_DS_FULL ? 8 : k == C_DQ_EMPTY || k == C_ACC_EMPTY ? 4 : 1;
      ptx::mbar_init(bars + k, n);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  for (int e = threadIdx.x; e < L::ZERO_BYTES / 16; e += blockDim.x)
    *(uint4*)(sm + L::ZERO_OFF + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
  // packed row tiles may leave rows that no copy ever writes: zeros, as 0 * NaN would be NaN
  if (p.s.packed)
    for (int e = threadIdx.x; e < (L::NQ + L::NDO) * L::TILE / 16; e += blockDim.x)
      *(uint4*)(sm + L::Q_OFF + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  if (warp == 1) ptx::tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  train::grid_wait();                              // Delta and LSE are there, the header is clear

  if (warp < 4) {
    ptx::regs_dec<L::REGS_SINGLE>();
    if (warp == 0 && lane == 0) {
      // ===================================== TMA producer =====================================
      BwdWalk w(p);
      int it = 0, tl = 0, loaded = 0;              // tasks, key tiles, dO tiles
      bool ok = !p.withhold;
      while (ok && w.next()) {
        const int qb = it % L::NQ;
        if (it >= L::NQ) ok = ptx::mbar_wait(bars + C_Q_EMPTY + qb, (it / L::NQ - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        const size_t row = ((size_t)w.bh * p.s.ntile + w.tile()) * kTile;
        uint8_t* offs = sm + L::OFFS_OFF + qb * L::OFFS;
        ptx::mbar_expect_tx(bars + C_Q_FULL + qb, row_tile_bytes<DT>(p.s) + L::OFFS);
        load_row_tile<DT>(p.s, &maps.q, sm + L::Q_OFF + qb * L::TILE, w.b, w.hk, w.tile(), p.s.q_b, p.s.q_h,
                          bars + C_Q_FULL + qb);
        ptx::bulk_load(offs, p.nnl + row, kTile * 4, bars + C_Q_FULL + qb);
        ptx::bulk_load(offs + kTile * 4, p.delta + row, kTile * 4, bars + C_Q_FULL + qb);
        if (w.first_of_tile()) {
          if (tl > 0) ok = ptx::mbar_wait(bars + C_KV_EMPTY, (tl - 1) & 1, abort_flag, tmo);
          if (!ok) {
            ++it;
            break;
          }
          ptx::mbar_expect_tx(bars + C_KV_FULL, 2 * L::TILE);
          load_key_tile<DT>(&maps.k, sm + L::K_OFF, w.b, w.hk, w.k0 + w.i, p.s.k_b, p.s.k_h, bars + C_KV_FULL);
          load_key_tile<DT>(&maps.v, sm + L::V_OFF, w.b, w.hk, w.k0 + w.i, p.s.v_b, p.s.v_h, bars + C_KV_FULL);
          ++tl;
        }
        const int ob = it % L::NDO;
        if (it >= L::NDO) ok = ptx::mbar_wait(bars + C_DO_EMPTY + ob, (it / L::NDO - 1) & 1, abort_flag, tmo);
        if (!ok) {
          ++it;
          break;
        }
        ptx::mbar_expect_tx(bars + C_DO_FULL + ob, row_tile_bytes<DT>(p.s));
        load_row_tile<DT>(p.s, &maps.dO, sm + L::DO_OFF + ob * L::TILE, w.b, w.hk, w.tile(), 1, 1,
                          bars + C_DO_FULL + ob);
        ++loaded;
        ++it;
        // the unit's first pass over its rows finds them in memory: ask for the tiles after the
        // buffered ones, so that they wait in L2
        if (w.i == 0 && w.j + L::NDO < w.nqt) {
          prefetch_row_tile<DT>(p.s, &maps.q, w.b, w.hk, w.tile() + L::NDO, p.s.q_b, p.s.q_h);
          prefetch_row_tile<DT>(p.s, &maps.dO, w.b, w.hk, w.tile() + L::NDO, 1, 1);
        }
      }
      // drain: every issued load has landed before the CTA may exit
      for (int k = max(0, it - L::NQ); k < it; ++k)
        ptx::mbar_drain(bars + C_Q_FULL + k % L::NQ, (k / L::NQ) & 1, 100000000ll);
      for (int k = max(0, loaded - L::NDO); k < loaded; ++k)
        ptx::mbar_drain(bars + C_DO_FULL + k % L::NDO, (k / L::NDO) & 1, 100000000ll);
      if (tl > 0) ptx::mbar_drain(bars + C_KV_FULL, (tl - 1) & 1, 100000000ll);
    } else if (warp == 2) {
      // ============================== key rows behind a length ================================
      BwdWalk w(p);
      int tl = 0;
      bool ok = true;
      while (ok && w.next()) {
        if (!w.first_of_tile()) continue;
        ok = ptx::warp_wait(bars + C_KV_FULL, tl & 1, abort_flag, tmo);
        if (!ok) break;
        if (w.keys() < kTile && w.len < p.s.Sk) {
          clear_rows<DT>(sm + L::K_OFF, w.keys(), kTile, lane);
          clear_rows<DT>(sm + L::V_OFF, w.keys(), kTile, lane);
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + C_KV_READY);
        ++tl;
      }
    } else if (warp == 1 && lane == 0) {
      // ===================================== MMA issuer =======================================
      const uint32_t sK = ptx::smem_u32(sm + L::K_OFF), sV = ptx::smem_u32(sm + L::V_OFF);
      const uint32_t sQ = ptx::smem_u32(sm + L::Q_OFF), sdO = ptx::smem_u32(sm + L::DO_OFF);
      const uint32_t sDS = ptx::smem_u32(sm + L::DS_OFF);
      const uint32_t dK_k = ptx::sdesc_lo(sK, 16), dV_k = ptx::sdesc_lo(sV, 16);
      const uint32_t dKt_mn = ptx::sdesc_lo(sK, DT == 128 ? kTile * 128 : L::ZERO_OFF - L::K_OFF);
      const uint32_t dQ_k0 = ptx::sdesc_lo(sQ, 16), dQ_mn0 = ptx::sdesc_lo(sQ, kTile * 128);
      const uint32_t ddO_k = ptx::sdesc_lo(sdO, 16), ddO_mn = ptx::sdesc_lo(sdO, kTile * 128);
      const uint32_t dDS_mn = ptx::sdesc_lo(sDS, kTile * 128);
      constexpr uint32_t ID_S = ptx::idesc_bf16(128, 128, 0, 0);
      const uint32_t id_ts = ptx::idesc_bf16(128, dsteps * 16, 0, 1);
      constexpr uint32_t ID_DQ = ptx::idesc_bf16(128, 128, 1, 1);
      constexpr uint32_t BUF_STEP = L::TILE >> 4;
      BwdWalk w(p);
      int it = 0, tile = -1;
      bool ok = true, have = w.next(), s_done = false;   // s_done: S(it) was issued ahead
      while (ok && have) {
        const bool first = w.first_of_tile(), last = w.last_of_tile();
        const int qb = it % L::NQ, ob = it % L::NDO, ksteps = (w.keys() + 15) >> 4;
        if (first) {
          ++tile;
          ok = ptx::mbar_wait(bars + C_KV_READY, tile & 1, abort_flag, tmo);
          if (!ok) break;
        }
        // ---- S^T(it), once Q(it) has landed and dK(it-1) has released the dS^T columns
        if (!s_done) {
          ok = ptx::mbar_wait(bars + C_Q_FULL + qb, (it / L::NQ) & 1, abort_flag, tmo);
          if (ok && it > 0) ok = ptx::mbar_wait(bars + C_SP_FREE, (it - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_SP, dK_k, dQ_k0 + qb * BUF_STEP, ID_S, dsteps);
          ptx::mma_commit(bars + C_S_FULL);
        }
        // ---- dP^T(it), once dO(it) has landed and dQ^T(it-1) has left the columns they share
        ok = ptx::mbar_wait(bars + C_DO_FULL + ob, (it / L::NDO) & 1, abort_flag, tmo);
        if (ok && !L::kSepDQ && it > 0) ok = ptx::mbar_wait(bars + C_DQ_EMPTY, (it - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_scores<DT>(tmem + L::T_DP, dV_k, ddO_k + ob * BUF_STEP, ID_S, dsteps);
        ptx::mma_commit(bars + C_DP_FULL);
        // ---- dV += P^T dO, once P^T(it) is stored and the last key tile's sums were read out
        ok = ptx::mbar_wait(bars + C_P_FULL, it & 1, abort_flag, tmo);
        if (ok && first && tile > 0) ok = ptx::mbar_wait(bars + C_ACC_EMPTY, (tile - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t acc0 = first ? 0u : 1u;
        issue_ts(tmem + L::T_DV, tmem + L::T_SP, ddO_mn + ob * BUF_STEP, id_ts, acc0);
        ptx::mma_commit(bars + C_DO_EMPTY + ob);
        have = w.next();
        // ---- dK += dS^T Q, then dQ^T = K^T dS^T, once dS^T(it) is stored
        ok = ptx::mbar_wait(bars + C_DS_FULL, it & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_ts(tmem + L::T_DK, tmem + L::T_SP + 32, dQ_mn0 + qb * BUF_STEP, id_ts, acc0);
        ptx::mma_commit(bars + C_Q_EMPTY + qb);
        ptx::mma_commit(bars + C_SP_FREE);
        // ---- S^T(it+1) of the same keys ahead of dQ^T(it) (DT = 64) or between its halves, so
        // that the softmax gradient has it earlier
        s_done = have && !w.first_of_tile();
        if (L::kSepDQ && it > 0) ok = ptx::mbar_wait(bars + C_DQ_EMPTY, (it - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        uint32_t dq_a = dKt_mn, dq_b = dDS_mn;
        if (DT == 128 && s_done) issue_dq<0, 4>(tmem + L::T_DQ, dq_a, dq_b, ID_DQ, ksteps);
        if (s_done) {
          const int qn = (it + 1) % L::NQ;
          ok = ptx::mbar_wait(bars + C_Q_FULL + qn, ((it + 1) / L::NQ) & 1, abort_flag, tmo);
          if (ok) ok = ptx::mbar_wait(bars + C_SP_FREE, it & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_SP, dK_k, dQ_k0 + qn * BUF_STEP, ID_S, dsteps);
          ptx::mma_commit(bars + C_S_FULL);
        }
        if (DT == 128 && s_done) issue_dq<4, 8>(tmem + L::T_DQ, dq_a, dq_b, ID_DQ, ksteps);
        else issue_dq<0, 8>(tmem + L::T_DQ, dq_a, dq_b, ID_DQ, ksteps);
        ptx::mma_commit(bars + C_DQ_FULL);
        if (last) {
          ptx::mma_commit(bars + C_ACC_FULL);
          ptx::mma_commit(bars + C_KV_EMPTY);
        }
        ++it;
      }
      // drain: no MMA may be in flight when TMEM is released
      ptx::mma_commit(bars + C_DRAIN);
      ptx::mbar_drain(bars + C_DRAIN, 0, 1000000000ll);
    }
  } else if (warp < 12) {
    // =============================== softmax-gradient warps =================================
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;             // key within the tile (TMEM lane)
    const int col0 = half * 64;                    // this thread's 64 rows
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    const uint32_t sDS = ptx::smem_u32(sm + L::DS_OFF);
    BwdWalk w(p);
    int it = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int qb = it % L::NQ;
      // (the offsets beside Q were copied by TMA: their own barrier is waited for as well)
      ok = ptx::warp_wait(bars + C_Q_FULL + qb, (it / L::NQ) & 1, abort_flag, tmo) &&
           ptx::warp_wait(bars + C_S_FULL, it & 1, abort_flag, tmo);
      if (!ok) break;
      ptx::tc_fence_after();
      const float* nnl = (const float*)(sm + L::OFFS_OFF + qb * L::OFFS) + col0;
      const float* delta = nnl + kTile;
      float pv[64];
      {
        uint32_t a[32], b[32];
        ptx::tmem_ld32_issue(tmem + lane_addr + L::T_SP + col0, a);
        ptx::tmem_ld32_wait(a);
        ptx::tmem_ld32_issue(tmem + lane_addr + L::T_SP + col0 + 32, b);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 f = *(const float4*)(nnl + c);
          pv[c] = ptx::ex2(fmaf(__uint_as_float(a[c]), p.scale_log2, f.x));
          pv[c + 1] = ptx::ex2(fmaf(__uint_as_float(a[c + 1]), p.scale_log2, f.y));
          pv[c + 2] = ptx::ex2(fmaf(__uint_as_float(a[c + 2]), p.scale_log2, f.z));
          pv[c + 3] = ptx::ex2(fmaf(__uint_as_float(a[c + 3]), p.scale_log2, f.w));
        }
        ptx::tmem_ld32_wait(b);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 f = *(const float4*)(nnl + 32 + c);
          pv[32 + c] = ptx::ex2(fmaf(__uint_as_float(b[c]), p.scale_log2, f.x));
          pv[33 + c] = ptx::ex2(fmaf(__uint_as_float(b[c + 1]), p.scale_log2, f.y));
          pv[34 + c] = ptx::ex2(fmaf(__uint_as_float(b[c + 2]), p.scale_log2, f.z));
          pv[35 + c] = ptx::ex2(fmaf(__uint_as_float(b[c + 3]), p.scale_log2, f.w));
        }
      }
      const bool dead = r >= w.keys();             // a key behind the length
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t u[8];
        if (dead) {
#pragma unroll
          for (int c = 16 * g; c < 16 * g + 16; ++c) pv[c] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = ptx::pack_bf16(pv[16 * g + 2 * k], pv[16 * g + 2 * k + 1]);
        ptx::tmem_st8(tmem + lane_addr + L::T_SP + col0 + 8 * g, u);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + C_P_FULL);
      // dP^T(it) is complete; its commit covers dQ^T(it-1), the last reader of the dS^T tile
      ok = ptx::warp_wait(bars + C_DP_FULL, it & 1, abort_flag, tmo);
      if (!ok) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 16) {
        float dp[16];
        ptx::tmem_ld16(tmem + lane_addr + L::T_DP + col0 + c0, dp);
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float4 f = *(const float4*)(delta + c0 + 2 * k);
          u[k] = ptx::pack_bf16(pv[c0 + 2 * k] * (dp[2 * k] - f.x), pv[c0 + 2 * k + 1] * (dp[2 * k + 1] - f.y));
          u[k + 1] = ptx::pack_bf16(pv[c0 + 2 * k + 2] * (dp[2 * k + 2] - f.z),
                                    pv[c0 + 2 * k + 3] * (dp[2 * k + 3] - f.w));
        }
        ptx::tmem_st8(tmem + lane_addr + L::T_SP + col0 + 32 + c0 / 2, u);
        store_chunk8(sDS, r, (col0 + c0) / 8, u);
        store_chunk8(sDS, r, (col0 + c0) / 8 + 1, u + 4);
      }
      ptx::tmem_wait_st();
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + C_DS_FULL);
      ++it;
    }
  } else {
    // ======================= dQ read-out, and the epilogue of dK and dV ======================
    ptx::regs_inc<L::REGS_READOUT>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;           // d of dQ^T; key of dK and dV
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    BwdWalk w(p);
    int it = 0, tl = 0;
    bool ok = true;
    while (ok && w.next()) {
      const bool holds = quarter * 32 < p.s.D;     // this warp's lanes are columns of dQ
      const bool begins = w.i == 0, ends = w.i == w.nkt - 1 && p.ksegs == 1;
      float* acc = p.dq_acc + ((((size_t)w.kseg * p.s.B * p.s.Hk + w.bh) * p.s.ntile + w.tile()) * kTile) * DT + 4 * row;
      // what the key tiles before added up to, for the last one: fetched while its products run
      float v[128];
      if (holds && ends && !begins) {
#pragma unroll
        for (int c = 0; c < 128; c += 4) ld_relaxed_v4(acc + (size_t)c * DT, v + c);
      } else {
#pragma unroll
        for (int c = 0; c < 128; ++c) v[c] = 0.f;
      }
      ok = ptx::warp_wait(bars + C_DQ_FULL, it & 1, abort_flag, tmo);
      if (!ok) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float t[32];
        ptx::tmem_ld32(tmem + lane_addr + L::T_DQ + c0, t);
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c0 + c] += t[c];
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + C_DQ_EMPTY);   // dQ^T(it) has left TMEM
      if (holds) {
        if (ends) {
          // Lanes 2k and 2k + 1 hold d = 2k and 2k + 1 of every row: the even lane takes both for
          // even rows, the odd lane for odd ones, so that a store has two of them.
          const int odd = lane & 1, d = row & ~1;
          int token, head;
          row_of(p.s, w.tile(), odd, token, head);
          __nv_bfloat16* dst = p.dq + w.b * p.dq_b + w.hk * p.s.g * p.dq_h + d;
          dst += token * p.dq_s + head * p.dq_h;
          uint32_t two[64];
#pragma unroll
          for (int c = 0; c < 128; c += 2) {
            const float give = odd ? v[c] : v[c + 1], keep = odd ? v[c + 1] : v[c];
            const float got = __shfl_xor_sync(0xffffffffu, give, 1);
            two[c / 2] = ptx::pack_bf16((odd ? got : keep) * p.scale, (odd ? keep : got) * p.scale);
          }
          if (d < p.s.D) {
            if (!p.s.packed) {
              const long long step = 2 * p.dq_s;
              const int left = p.s.Sq - token;
#pragma unroll
              for (int c = 0; c < 128; c += 2) {
                if (c < left) *reinterpret_cast<uint32_t*>(dst) = two[c / 2];
                dst += step;
              }
            } else {
              int left = min(p.s.tpt, p.s.Sq - token);
#pragma unroll
              for (int c = 0; c < 128; c += 2) {
                if (left > 0) *reinterpret_cast<uint32_t*>(dst) = two[c / 2];
                head += 2;                         // two heads on, or into the next token
                dst += 2 * p.dq_h;
                if (head >= p.s.g) {
                  head -= p.s.g;
                  dst += p.dq_s - p.s.g * p.dq_h;
                  --left;
                }
              }
            }
          }
        } else if (!begins) {
#pragma unroll
          for (int c = 0; c < 128; c += 4)
            ptx::red_add_v4_f32(acc + (size_t)c * DT, v[c], v[c + 1], v[c + 2], v[c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 4)
            *(float4*)(acc + (size_t)c * DT) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
      }
      if (w.last_of_tile()) {
        ok = ptx::warp_wait(bars + C_ACC_FULL, tl & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        const int kt = w.k0 + w.i, key = kt * kTile + row;
        float* part = p.dkv_part + ((((size_t)w.qseg * p.s.B * p.s.Hk + w.bh) * p.s.nk + kt) * 2 * kTile + row) * DT;
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // dK, then dV
          const uint32_t from = tmem + lane_addr + (which ? L::T_DV : L::T_DK);
          __nv_bfloat16* dst = which ? p.dv + w.b * p.dv_b + key * p.dv_s + w.hk * p.dv_h
                                     : p.dk + w.b * p.dk_b + key * p.dk_s + w.hk * p.dk_h;
#pragma unroll
          for (int c0 = 0; c0 < DT; c0 += 32) {
            if (c0 < p.s.D) {
              float a[32];
              ptx::tmem_ld32(from + c0, a);
              if (p.qsegs > 1) {
                float4* d4 = (float4*)(part + which * kTile * DT + c0);
#pragma unroll
                for (int k = 0; k < 8; ++k) d4[k] = make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
              } else if (key < p.s.Sk) {
                store_bf16_32(dst + c0, a, which ? 1.f : p.scale, p.s.D - c0);
              }
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + C_ACC_EMPTY);
        ++tl;
      }
      ++it;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicCAS(p.header + WS_STATUS, 0, kStatusSyncTimeout);
}

// What the units left: dq as the sum of the key segments' partials, dk and dv as that of the row
// segments', in order; zeros where no key was visible, NaN for a length out of range. The first
// dq_blocks blocks take a row tile each, 16 rows at a time through shared memory, as the partials
// hold four rows of a column side by side; a thread of the others 8 columns of a row.
template <int DT>
__global__ void __launch_bounds__(256) cross_grad_join_kernel(const __grid_constant__ BwdArgs p, unsigned dq_blocks) {
  __shared__ float rows16[16][DT + 4];
  train::grid_wait();
  const size_t groups = (size_t)p.s.B * p.s.Hk;
  float t[8];
  if (blockIdx.x < dq_blocks) {
    const size_t tile_id = blockIdx.x;             // group, tile
    const int tile = (int)(tile_id % p.s.ntile), bh = (int)(tile_id / p.s.ntile);
    const int b = bh / p.s.Hk, hk = bh - b * p.s.Hk;
    const int len = length_of(p.s, b), tiles = (max(len, 0) + kTile - 1) / kTile;
    if (len > 0 && p.ksegs == 1) return;           // written by the one unit of these rows
    const int n = (tiles + p.kper - 1) / p.kper;
    const size_t step = groups * p.s.ntile * kTile * DT;
    for (int r0 = 0; r0 < kTile; r0 += 16) {
      const float* src = p.dq_acc + (tile_id * kTile + r0) * DT;
      for (int e = threadIdx.x; e < 4 * DT; e += 256) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < n; ++s) {
          const float4 y = __ldg((const float4*)(src + s * step) + e);
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        const int q = e / DT * 4, d = e % DT;
        rows16[q][d] = x.x;
        rows16[q + 1][d] = x.y;
        rows16[q + 2][d] = x.z;
        rows16[q + 3][d] = x.w;
      }
      __syncthreads();
      const int r = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;
      int token, head;
      if (c < p.s.D && row_of(p.s, tile, r0 + r, token, head)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = len < 0 ? NAN : rows16[r][c + i] * p.scale;
        train::store_f32<__nv_bfloat16, 8>(p.dq + b * p.dq_b + token * p.dq_s + (hk * p.s.g + head) * p.dq_h + c, t);
      }
      __syncthreads();
    }
    return;
  }
  const int per = p.s.D >> 3;
  const long long item = (long long)(blockIdx.x - dq_blocks) * 256 + threadIdx.x;
  const int c = (int)(item % per) * 8;
  const long long row = item / per;                // (batch, key, head)
  if (row >= (long long)p.s.B * p.s.Sk * p.s.Hk) return;
  const int h = (int)(row % p.s.Hk);
  const int token = (int)(row / p.s.Hk % p.s.Sk), b = (int)(row / p.s.Hk / p.s.Sk);
  const int len = length_of(p.s, b), tiles = (max(len, 0) + kTile - 1) / kTile;
  const int kt = token / kTile;
  if (kt < tiles && p.qsegs == 1) return;
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = len < 0 ? NAN : 0.f;
    if (kt < tiles) {
      const float* src = p.dkv_part + ((((size_t)b * p.s.Hk + h) * p.s.nk + kt) * 2 * kTile + which * kTile + token % kTile) * DT + c;
      const size_t step = groups * p.s.nk * 2 * kTile * DT;
      for (int s = 0; s < p.qsegs; ++s) {
        float x[8];
        train::load_f32<float, 8>(src + s * step, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] += x[i];
      }
      if (!which)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= p.scale;
    }
    __nv_bfloat16* dst = which ? p.dv + b * p.dv_b + token * p.dv_s + h * p.dv_h
                               : p.dk + b * p.dk_b + token * p.dk_s + h * p.dk_h;
    train::store_f32<__nv_bfloat16, 8>(dst + c, t);
  }
}

}  // namespace cross
}  // namespace dash
