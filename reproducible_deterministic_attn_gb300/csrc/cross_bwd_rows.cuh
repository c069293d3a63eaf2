// Cross attention backward, dQ = scale dS K of groups with several key tiles. A unit of work is a
// row tile of a group and a range of its key tiles; a persistent grid takes the units in turn. The
// row tile's Q and dO stay in shared memory, and dQ accumulates in TMEM, over the key tiles:
//   S   = Q K^T       M = 128 rows, N = the tile's keys, K = D       TMEM cols [128 b, +128), b = t % 2
//   dP  = dO V^T      M = 128 rows, N = the tile's keys, K = D       TMEM cols [256, +128)
//   dS  = P * (dP - Delta), P = exp2(S scale log2e - LSE log2e)      bf16, TMEM, over S's columns
//   dQ += dS K        M = 128 rows, N = D, K = the tile's keys       TMEM cols [384, +DT), A from TMEM
// S(t+1) is computed while the softmax gradient works on t, dP(t+1) goes ahead of dQ(t), S(t+2)
// follows dQ(t). LSE and Delta are one number a thread here, as a thread owns a row (and half of the
// keys). Key ranges (few row tiles against many keys) leave fp32 partials that
// cross_join_rows_kernel adds in order. A key tile takes 1 us, where the products take 1536 cycles
// and shared memory 1800 (two products with both operands there, K and V copied in).
//
// A unit of few key tiles (a text) lasts little longer than its ends, which the next one's copies run
// under: Q's under the last dP, dO's under the last dQ (8192 x 512, 16 heads of 128: 94 us, before both
// waited for the last dP, then 86, now 81; warps of their own for the read-out of dQ gained nothing).
//
// Warp roles (384 threads): 0 = TMA producer, 1 and 3 = MMA issuers (S; dP and dQ), 2 = K rows
// behind a length, 4..11 = softmax gradient (quarter = TMEM lanes = rows, half = 64 keys each) and
// the epilogue. Every wait is bounded.
#pragma once

#include "cross_bwd.cuh"

namespace dash {
namespace cross {

template <int DT>
struct RowsLay {
  static constexpr int TILE = kTile * DT * 2;
  static constexpr int NB = DT == 64 ? 2 : 1;                  // Q and dO buffers
  // K waits for dQ, V only for dP: so K has more stages
  static constexpr int KST = DT == 64 ? 5 : 3, VST = DT == 64 ? 4 : 2;
  static constexpr int Q_OFF = 0, K_OFF = 2 * NB * TILE;       // buffer b: Q, dO
  static constexpr int V_OFF = K_OFF + KST * TILE;
  static constexpr int BAR_OFF = V_OFF + VST * TILE;
  static constexpr int ALLOC = BAR_OFF + 512 + 1024;           // slack for 1024 alignment
  static_assert(ALLOC <= 232448, "shared memory budget");
  static constexpr int T_S = 0, T_DP = 256, T_DQ = 384;
  static constexpr int Q_FULL = 0, DO_FULL = NB, Q_EMPTY = 2 * NB, DO_EMPTY = 3 * NB, S_FULL = 4 * NB, S_FREE = S_FULL + 2,
                       DP_FULL = S_FREE + 2, DS_FULL = DP_FULL + 1, ACC_FULL = DS_FULL + 1,
                       ACC_EMPTY = ACC_FULL + 1, DRAIN = ACC_EMPTY + 1, K_FULL = DRAIN + 2,
                       V_FULL = K_FULL + KST, K_EMPTY = V_FULL + VST, V_EMPTY = K_EMPTY + KST,
                       CLEAN = V_EMPTY + VST, COUNT = CLEAN + KST;
  static_assert(8 * COUNT + 8 <= 512, "barrier area");
};
constexpr int kRowsThreads = 384;
constexpr int kRowsRegsLaunch = 168, kRowsRegsCtrl = 88, kRowsRegsSoftmax = 208;
static_assert(kRowsRegsCtrl + 2 * kRowsRegsSoftmax == 3 * kRowsRegsLaunch,
              "the three warpgroups must share exactly the launch's registers");

// A CTA's units, [batch][row tile][key head][key range]; those without keys are passed over
// (cross_pre_kernel writes their rows, and the join reads no range behind a length). ALL: a whole
// warp walks together.
template <bool ALL = false>
struct RowsWalk {
  const BwdArgs* a;
  Place at;                  // d0: key range, d1: row tile
  int known, len;            // the batch whose length is at hand (-2: not begun), that length
  int t0, nt;                // first key tile and their number in this range
  __device__ __forceinline__ RowsWalk(const BwdArgs& args)
      : a(&args), at(args.units), known(-2), len(0) {}
  __device__ __forceinline__ bool next() {
    const BwdArgs& p = *a;
    do {
      if (known == -2) known = -1;
      else at.next(p.units);
      if (!at.more(p.units)) return false;
      if (at.b != known) {
        known = at.b;
        len = length_of(p.s, known);
        if (ALL) len = same(len);
      }
      t0 = at.d0 * p.kper;
      nt = min((max(len, 0) + kTile - 1) / kTile, t0 + p.kper) - t0;
    } while (nt <= 0);
    return true;
  }
  __device__ __forceinline__ int group() const { return at.b * a->s.Hk + at.hk; }
  __device__ __forceinline__ int keys(int t) const { return min(kTile, len - (t0 + t) * kTile); }
  __device__ __forceinline__ int steps(int t) const { return (keys(t) + 15) >> 4; }   // of 16 keys
  // rows of the K tile that dQ reads although the length leaves them out
  __device__ __forceinline__ bool unclean(int t) const { return len < a->s.Sk && (keys(t) & 15); }
};

template <int DT>
__global__ void __launch_bounds__(kRowsThreads, 1)
    cross_rows_kernel(const __grid_constant__ BwdArgs p, const __grid_constant__ Maps maps) {
  using L = RowsLay<DT>;
  extern __shared__ uint8_t smem_crossr[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_crossr + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(sm + L::BAR_OFF);
  uint32_t* tmem_slot = (uint32_t*)(sm + L::BAR_OFF + 8 * L::COUNT);
  volatile int* abort_flag = (volatile int*)(sm + L::BAR_OFF + 8 * L::COUNT + 4);
  const int warp = same((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const long long tmo = p.timeout_ns;
  const int dsteps = (p.s.D + 15) >> 4;

  train::grid_next();
  if (threadIdx.x == 0) {
    for (int k = 0; k < L::COUNT; ++k) {
      const bool key = k >= L::K_EMPTY && k < L::V_EMPTY;   // the products, and warp 2
      ptx::mbar_init(bars + k, k == L::DS_FULL || k == L::ACC_EMPTY ? 8 : key && p.s.lens ? 2 : 1);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);
  train::grid_wait();                              // Delta and LSE are there, the header is clear

  if (warp < 4) {
    ptx::regs_dec<kRowsRegsCtrl>();
    if (warp == 0 && lane == 0) {
      // ===================================== TMA producer =====================================
      RowsWalk<> w(p);
      int n = 0, kv = 0, nk = 0, nd = 0;           // units, key tiles (V), K tiles, dO tiles so far
      bool ok = !p.withhold;
      while (ok && w.next()) {
        const int b = n % L::NB;
        if (n >= L::NB) ok = ptx::mbar_wait(bars + L::Q_EMPTY + b, (n / L::NB - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        uint8_t* q = sm + L::Q_OFF + 2 * b * L::TILE;
        ptx::mbar_expect_tx(bars + L::Q_FULL + b, row_tile_bytes<DT>(p.s));
        load_row_tile<DT>(p.s, &maps.q, q, w.at.b, w.at.hk, w.at.d1, p.s.q_b, p.s.q_h, bars + L::Q_FULL + b);
        for (int t = 0; ok && t < w.nt; ++t, ++kv) {
          const int ks = kv % L::KST, km = kv / L::KST, vs = kv % L::VST, vm = kv / L::VST;
          if (km > 0) ok = ptx::mbar_wait(bars + L::K_EMPTY + ks, (km - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::K_FULL + ks, L::TILE);
          load_key_tile<DT>(&maps.k, sm + L::K_OFF + ks * L::TILE, w.at.b, w.at.hk, w.t0 + t, p.s.k_b, p.s.k_h,
                            bars + L::K_FULL + ks);
          ++nk;
          if (t == 0) {
            // Q is free before dO is (the last S goes ahead of the last dP), so that the next unit's
            // first S is there when this one's rows have left
            if (n >= L::NB) ok = ptx::mbar_wait(bars + L::DO_EMPTY + b, (n / L::NB - 1) & 1, abort_flag, tmo);
            if (!ok) break;
            ptx::mbar_expect_tx(bars + L::DO_FULL + b, row_tile_bytes<DT>(p.s));
            load_row_tile<DT>(p.s, &maps.dO, q + L::TILE, w.at.b, w.at.hk, w.at.d1, 1, 1, bars + L::DO_FULL + b);
            ++nd;
          }
          if (vm > 0) ok = ptx::mbar_wait(bars + L::V_EMPTY + vs, (vm - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::V_FULL + vs, L::TILE);
          load_key_tile<DT>(&maps.v, sm + L::V_OFF + vs * L::TILE, w.at.b, w.at.hk, w.t0 + t, p.s.v_b, p.s.v_h,
                            bars + L::V_FULL + vs);
        }
        ++n;
      }
      // drain: every issued load has landed before the CTA may exit
      for (int k = max(0, n - L::NB); k < n; ++k)
        ptx::mbar_drain(bars + L::Q_FULL + k % L::NB, (k / L::NB) & 1, 100000000ll);
      for (int k = max(0, nd - L::NB); k < nd; ++k)
        ptx::mbar_drain(bars + L::DO_FULL + k % L::NB, (k / L::NB) & 1, 100000000ll);
      for (int k = max(0, nk - L::KST); k < nk; ++k)
        ptx::mbar_drain(bars + L::K_FULL + k % L::KST, (k / L::KST) & 1, 100000000ll);
      for (int k = max(0, kv - L::VST); k < kv; ++k)
        ptx::mbar_drain(bars + L::V_FULL + k % L::VST, (k / L::VST) & 1, 100000000ll);
    } else if (warp == 1) {
      // ===================================== issuer of S ======================================
      const uint32_t sQ = ptx::smem_u32(sm + L::Q_OFF), sK = ptx::smem_u32(sm + L::K_OFF);
      constexpr uint32_t TILE16 = L::TILE >> 4;
      RowsWalk<true> w(p);
      const uint32_t one = elect_one();
      int n = 0, k = 0;                            // units and key tiles so far
      bool ok = true;
      while (ok && w.next()) {
        const int b = n % L::NB;
        const uint32_t dQ = ptx::sdesc_lo(sQ, 16) + 2 * b * TILE16;
        ok = ptx::warp_wait(bars + L::Q_FULL + b, (n / L::NB) & 1, abort_flag, tmo);
        for (int t = 0; ok && t < w.nt; ++t, ++k) {
          // K(t) has landed, the buffer's last dS has been read by its dQ product
          const int s = k % L::KST;
          ok = ptx::warp_wait(bars + L::K_FULL + s, (k / L::KST) & 1, abort_flag, tmo);
          if (ok && k >= 2) ok = ptx::warp_wait(bars + L::S_FREE + (k & 1), (k / 2 - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_S + 128 * (k & 1), dQ, ptx::sdesc_lo(sK, 16) + s * TILE16,
                           ptx::idesc_bf16(128, 16 * w.steps(t), 0, 0), dsteps, one);
          commit(bars + L::S_FULL + (k & 1), one);
        }
        commit(bars + L::Q_EMPTY + b, one);
        ++n;
      }
      commit(bars + L::DRAIN, one);
      ptx::mbar_drain(bars + L::DRAIN, 0, 1000000000ll);
    } else if (warp == 3) {
      // ================================= issuer of dP and dQ ==================================
      const uint32_t sQ = ptx::smem_u32(sm + L::Q_OFF), sK = ptx::smem_u32(sm + L::K_OFF);
      const uint32_t sV = ptx::smem_u32(sm + L::V_OFF);
      const uint32_t id_dq = ptx::idesc_bf16(128, dsteps * 16, 0, 1);
      constexpr uint32_t TILE16 = L::TILE >> 4;
      RowsWalk<true> w(p);
      const uint32_t one = elect_one();
      int n = 0, k0 = 0;                           // units and key tiles before this unit
      uint32_t clean = 0;                          // parities of the stages' CLEAN barriers
      bool ok = true;
      while (ok && w.next()) {
        const int b = n % L::NB;
        const uint32_t ddO = ptx::sdesc_lo(sQ, 16) + (2 * b + 1) * TILE16;
        // dP(t): its columns were read when dS(t-1) was stored
        auto issue_dp = [&](int t, bool landed) {
          const int k = k0 + t, s = k % L::VST;
          if (!landed && !ptx::warp_wait(bars + L::V_FULL + s, (k / L::VST) & 1, abort_flag, tmo)) return false;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_DP, ddO, ptx::sdesc_lo(sV, 16) + s * TILE16,
                           ptx::idesc_bf16(128, 16 * w.steps(t), 0, 0), dsteps, one);
          commit(bars + L::DP_FULL, one);
          commit(bars + L::V_EMPTY + s, one);
          if (t == w.nt - 1) commit(bars + L::DO_EMPTY + b, one);
          return true;
        };
        ok = ptx::warp_wait(bars + L::DO_FULL + b, (n / L::NB) & 1, abort_flag, tmo) && issue_dp(0, false);
        for (int t = 0; ok && t < w.nt; ++t) {
          const int k = k0 + t, s = k % L::KST;
          // the rest of what the products wait for comes before, out of the way from dS to them
          const int vk = k + 1, vs = vk % L::VST;
          const bool landed = t + 1 < w.nt && is_complete(bars + L::V_FULL + vs, (vk / L::VST) & 1);
          ok = ptx::warp_wait(bars + L::K_FULL + s, (k / L::KST) & 1, abort_flag, tmo);
          if (ok && t == 0 && n > 0) ok = ptx::warp_wait(bars + L::ACC_EMPTY, (n - 1) & 1, abort_flag, tmo);
          if (ok && t == w.nt - 1 && w.unclean(t)) {
            ok = ptx::warp_wait(bars + L::CLEAN + s, (clean >> s) & 1, abort_flag, tmo);
            clean ^= 1u << s;
          }
          if (ok) ok = ptx::warp_wait(bars + L::DS_FULL, k & 1, abort_flag, tmo);
          if (ok && t + 1 < w.nt) ok = issue_dp(t + 1, landed);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t dK = ptx::sdesc_lo(sK + s * L::TILE, kTile * 128);
          issue_rows<true>(tmem + L::T_DQ, tmem + L::T_S + 128 * (k & 1), dK, id_dq, t > 0 ? 1u : 0u, w.steps(t), one);
          commit(bars + L::S_FREE + (k & 1), one);
          commit(bars + L::K_EMPTY + s, one);
        }
        if (!ok) break;
        commit(bars + L::ACC_FULL, one);
        k0 += w.nt;
        ++n;
      }
      commit(bars + L::DRAIN + 1, one);
      ptx::mbar_drain(bars + L::DRAIN + 1, 0, 1000000000ll);
    } else if (warp == 2 && p.s.lens) {
      // ============================ rows of K behind a sequence's end ==========================
      // Every tile is waited for and its stage released here too, so that this warp can be neither
      // ahead of the copies nor behind the products by more than a barrier's phase.
      RowsWalk<> w(p);
      int kv = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int t = 0; t < w.nt; ++t, ++kv) {
          const int s = kv % L::KST;
          ok = ptx::warp_wait(bars + L::K_FULL + s, (kv / L::KST) & 1, abort_flag, tmo);
          if (!ok) break;
          if (t == w.nt - 1 && w.unclean(t)) {
            clear_rows<DT>(sm + L::K_OFF + s * L::TILE, w.keys(t), 16 * w.steps(t), lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bars + L::CLEAN + s);
          }
          if (lane == 0) ptx::mbar_arrive(bars + L::K_EMPTY + s);
        }
      }
    }
  } else {
    ptx::regs_inc<kRowsRegsSoftmax>();
    // ================================== softmax gradient ====================================
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;             // row within the tile = TMEM lane
    const int col0 = half * 64;                    // this thread's 64 keys
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    RowsWalk<> w(p);
    int n = 0, k = 0;                              // units, key tiles so far
    bool ok = true, more = w.next();
    float nnl, delta;                              // the row's -LSE log2e and -Delta
    auto fetch = [&]() {
      const size_t row = ((size_t)w.group() * p.s.ntile + w.at.d1) * kTile + r;
      nnl = __ldg(p.nnl + row);
      delta = __ldg(p.delta + row);
    };
    if (more) fetch();
    while (ok && more) {
      const uint64_t scale2 = two(p.scale_log2, p.scale_log2), nnl2 = two(nnl, nnl), delta2 = two(delta, delta);
      for (int t = 0; t < w.nt; ++t, ++k) {
        const uint32_t t_s = tmem + lane_addr + L::T_S + 128 * (k & 1) + col0;
        const int mine = 16 * w.steps(t) - col0;   // columns of this half that the products take
        ok = ptx::warp_wait(bars + L::S_FULL + (k & 1), (k >> 1) & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        float pv[64];
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          if (c0 < mine) {
            float x[32];
            ptx::tmem_ld32(t_s + c0, x);
#pragma unroll
            for (int c = 0; c < 32; c += 2) exp2_two(x[c], x[c + 1], scale2, nnl2, pv[c0 + c], pv[c0 + c + 1]);
          }
        }
        ok = ptx::warp_wait(bars + L::DP_FULL, k & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        const int live = w.keys(t) - col0;         // keys of this half
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          if (c0 < mine) {
            float dp[32];
            ptx::tmem_ld32(tmem + lane_addr + L::T_DP + col0 + c0, dp);
            uint32_t u[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              untwo(mul2(two(pv[c0 + c], pv[c0 + c + 1]), add2(two(dp[c], dp[c + 1]), delta2)), dp[c], dp[c + 1]);
            if (c0 + 32 > live) {                  // the sequence ends in here
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c >= live) dp[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) u[c] = ptx::pack_bf16(dp[2 * c], dp[2 * c + 1]);
            ptx::tmem_st8(t_s + c0 / 2, u);
            ptx::tmem_st8(t_s + c0 / 2 + 8, u + 8);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + L::DS_FULL);
      }
      if (!ok) break;
      ok = ptx::warp_wait(bars + L::ACC_FULL, n & 1, abort_flag, tmo);
      if (!ok) break;
      ptx::tc_fence_after();
      int token, head;
      const bool live = row_of(p.s, w.at.d1, r, token, head);
      __nv_bfloat16* dst = p.dq + w.at.b * p.dq_b + token * p.dq_s + (w.at.hk * p.s.g + head) * p.dq_h;
      float* part = p.dq_part + ((((size_t)w.at.d0 * p.s.B * p.s.Hk + w.group()) * p.s.ntile + w.at.d1) * kTile) * DT;
      more = w.next();
      if (more) fetch();                           // the next unit's, while this one's rows leave
#pragma unroll
      for (int i = 0; i < DT / 2; i += 32) {
        const int c0 = half * (DT / 2) + i;
        if (c0 < p.s.D) {
          float v[32];
          ptx::tmem_ld32(tmem + lane_addr + L::T_DQ + c0, v);
          if (p.ksegs == 1) store_rows_bf16(lane, v, p.scale, live ? dst + c0 : nullptr, p.s.D - c0);
          else if (live) store_part_32(part, r, c0, v, 1.f);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + L::ACC_EMPTY);
      ++n;
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

// dq as the sum of the key ranges' partials, in order; a thread takes 8 columns of a row.
template <int DT>
__global__ void __launch_bounds__(256) cross_join_rows_kernel(const __grid_constant__ BwdArgs p) {
  train::grid_next();
  train::grid_wait();
  const int per = p.s.D >> 3;
  const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
  const int c = (int)(item % per) * 8;
  const long long row = item / per;                // in row tiles
  const size_t rows = (size_t)p.s.B * p.s.Hk * p.s.ntile * kTile;
  if (row >= (long long)rows) return;
  const int r = (int)(row % kTile);
  const long long rest = row / kTile;
  const int tile = (int)(rest % p.s.ntile), bh = (int)(rest / p.s.ntile), b = bh / p.s.Hk, hk = bh - b * p.s.Hk;
  int token, head;
  if (!row_of(p.s, tile, r, token, head)) return;
  const int len = length_of(p.s, b);
  if (len <= 0) return;                            // written by cross_pre_kernel
  const int n = ((len + kTile - 1) / kTile + p.kper - 1) / p.kper;
  const float* src = p.dq_part + (size_t)(row - r) * DT + part_at(r, c);
  float t[8] = {};
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    float x[8];
    train::load_f32<float, 8>(src + s * rows * DT, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] += x[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] *= p.scale;
  train::store_f32<__nv_bfloat16, 8>(p.dq + b * p.dq_b + token * p.dq_s + (hk * p.s.g + head) * p.dq_h + c, t);
}

}  // namespace cross
}  // namespace dash
