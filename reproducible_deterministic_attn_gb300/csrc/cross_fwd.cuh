// Cross attention forward: O = softmax(scale Q K^T over the batch's keys) V and the natural-log
// LSE per row, on the 5th-generation tensor cores.
//
// A unit of work is a pair of row tiles (A and B) of one group of heads and a range of key tiles;
// a persistent grid runs the units in turn. Each row tile has a softmax warpgroup and TMEM of its
// own, both walk the same key tiles:
//   S_x = Q_x K_j^T       M = 128 rows, N = the tile's keys, K = D      TMEM cols [128 x, +128)
//   P_x = exp2(S_x scale log2e - m)      packed bf16: over S_x's first 64 columns (DT = 128) or in
//                                        64 columns of its own (DT = 64)
//   O_x += P_x V_j        M = 128, N = D, K = the tile's keys           TMEM cols [256 + DT x, +DT)
// While one warpgroup turns S into P the products of the other run, and while a unit's rows leave
// for memory the next unit's tiles load and its first S is computed. The last key tile of a
// sequence takes only its 32-column chunks with keys (77 keys: 96 columns, not 128).
// A softmax thread owns a row: it takes the row's scores out of TMEM once, so the maximum and the
// exponentials need no second read, and moves the exponent's reference m only when the row
// maximum exceeds it by more than 8 in log2 units (P <= 2^8; O and l share the reference).
//
// Key ranges (splits > 1): where the pairs of row tiles would leave most of the chip idle (single
// tokens against long states) the keys are cut into ranges; a range leaves its rows' normalised O
// in fp32 and their LSE, which cross_join_kernel combines in order.
//
// Warp roles (384 threads): 0 = TMA producer, 1 = MMA issuer, 2 = clears V rows that a length
// leaves out, 4..7 = softmax of tile A, 8..11 = of tile B. Every wait is bounded; a CTA that gives
// up writes NaN into the LSE of its rows and records DASH_ERR_SYNC_TIMEOUT where asked to.
#pragma once

#include "cross_common.cuh"

namespace dash {
namespace cross {

struct FwdArgs {
  Shape s;
  __nv_bfloat16* o;          // [B, Sq, Hq, D]
  float* lse;                // [B, Hq, Sq]
  float* part_o;             // splits > 1: [split][group][tile][128][DT]
  float* part_l;             //             [split][group][tile][128] LSE in log2 units
  int pairs, splits, kper;   // pairs of row tiles a group; key ranges, key tiles a range
  int units;
  float scale_log2;
  int* status;
  long long timeout_ns;
  int withhold;              // testing hook: load no keys, so that the waits for them run out
};

template <int DT>
struct FwdLay {
  static constexpr int TILE = kTile * DT * 2;
  static constexpr int STAGES = DT == 64 ? 4 : 2;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TILE;                     // stage s: K, then V
  static constexpr int BAR_OFF = KV_OFF + 2 * STAGES * TILE;
  static constexpr int ALLOC = BAR_OFF + 512 + 1024;          // slack for 1024 alignment
  static_assert(ALLOC <= 232448, "shared memory budget");
  static constexpr int T_S = 0, T_O = 256;
  static constexpr bool kSepP = DT == 64;                     // P in columns of its own
  static constexpr int T_P = kSepP ? T_O + 2 * DT : T_S;
  static constexpr int P_STRIDE = kSepP ? 64 : 128;
  static_assert(T_O + 2 * DT + (kSepP ? 128 : 0) <= 512, "TMEM columns");
  // barriers
  static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 6, PV_DONE = 8, DRAIN = 10,
                       K_FULL = 11, V_FULL = K_FULL + STAGES, KV_EMPTY = V_FULL + STAGES,
                       CLEAN = KV_EMPTY + STAGES, COUNT = CLEAN + STAGES;
  static_assert(8 * COUNT + 8 <= 512, "barrier area");
};

constexpr int kFwdThreads = 384;
constexpr float kRescaleLog2 = 8.f;
constexpr int kFwdRegsLaunch = 168, kFwdRegsCtrl = 88, kFwdRegsSoftmax = 208;
static_assert(kFwdRegsCtrl + 2 * kFwdRegsSoftmax == 3 * kFwdRegsLaunch,
              "the three warpgroups must share exactly the launch's registers");

// A CTA's units: u, u + grid, ... Every role walks the same ones.
struct FwdWalk {
  const FwdArgs& p;
  int u, bh, b, hk, pair, split;
  int len;                   // the batch's keys (-1: out of range)
  int t0, nt;                // first key tile and their number in this range
  bool has_b;
  __device__ __forceinline__ FwdWalk(const FwdArgs& a) : p(a), u((int)blockIdx.x - (int)gridDim.x) {}
  __device__ __forceinline__ bool next() {
    u += gridDim.x;
    if (u >= p.units) return false;
    split = u % p.splits;
    const int r = u / p.splits;
    pair = r % p.pairs;
    bh = r / p.pairs;
    b = bh / p.s.Hk;
    hk = bh - b * p.s.Hk;
    has_b = 2 * pair + 1 < p.s.ntile;
    len = length_of(p.s, b);
    t0 = split * p.kper;
    const int all = (max(len, 0) + kTile - 1) / kTile;
    nt = max(0, min(all, t0 + p.kper) - t0);
    return true;
  }
  // Keys of key tile t of this range, and how many 32-column chunks they take.
  __device__ __forceinline__ int keys(int t) const { return min(kTile, len - (t0 + t) * kTile); }
  __device__ __forceinline__ int chunks(int t) const { return (keys(t) + 31) >> 5; }
  // Rows of the V tile that the product reads although the length leaves them out (rows beyond
  // the tensor arrive as zeros).
  __device__ __forceinline__ bool unclean(int t) const { return len < p.s.Sk && (keys(t) & 31); }
};

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(ptx::smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

template <int DT>
__global__ void __launch_bounds__(kFwdThreads, 1)
    cross_fwd_kernel(const __grid_constant__ FwdArgs p, const __grid_constant__ Maps maps) {
  using L = FwdLay<DT>;
  extern __shared__ uint8_t smem_cross[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_cross + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(sm + L::BAR_OFF);
  uint32_t* tmem_slot = (uint32_t*)(sm + L::BAR_OFF + 8 * L::COUNT);
  volatile int* abort_flag = (volatile int*)(sm + L::BAR_OFF + 8 * L::COUNT + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long tmo = p.timeout_ns;
  const int dsteps = (p.s.D + 15) >> 4;

  if (p.splits > 1) train::grid_next();
  if (threadIdx.x == 0) {
    if (p.s.nk > 0) {
      ptx::prefetch_map(&maps.q);
      ptx::prefetch_map(&maps.k);
      ptx::prefetch_map(&maps.v);
    }
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(bars + L::Q_FULL + x, 1);
      ptx::mbar_init(bars + L::Q_EMPTY + x, 1);
      ptx::mbar_init(bars + L::S_FULL + x, 1);
      ptx::mbar_init(bars + L::P_FULL + x, 4);
      ptx::mbar_init(bars + L::PV_DONE + x, 1);
    }
    for (int s = 0; s < L::STAGES; ++s) {
      ptx::mbar_init(bars + L::K_FULL + s, 1);
      ptx::mbar_init(bars + L::V_FULL + s, 1);
      ptx::mbar_init(bars + L::KV_EMPTY + s, p.s.lens ? 2 : 1);   // the products, and warp 2
      ptx::mbar_init(bars + L::CLEAN + s, 1);
    }
    ptx::mbar_init(bars + L::DRAIN, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    ptx::regs_dec<kFwdRegsCtrl>();
    if (warp == 0 && lane == 0) {
      // ===================================== TMA producer =====================================
      FwdWalk w(p);
      int nqx[2] = {0, 0}, kv = 0;                 // row tiles and key tiles loaded so far
      bool ok = true;
      while (ok && w.next()) {
        if (w.nt == 0) continue;
        for (int x = 0; ok && x < (w.has_b ? 2 : 1); ++x) {
          if (nqx[x] > 0) ok = ptx::mbar_wait(bars + L::Q_EMPTY + x, (nqx[x] - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::Q_FULL + x, row_tile_bytes<DT>(p.s));
          load_row_tile<DT>(p.s, &maps.q, sm + L::Q_OFF + x * L::TILE, w.b, w.hk, 2 * w.pair + x, p.s.q_b, p.s.q_h,
                            bars + L::Q_FULL + x);
          ++nqx[x];
        }
        for (int t = 0; ok && t < (p.withhold ? 0 : w.nt); ++t, ++kv) {
          const int s = kv % L::STAGES, n = kv / L::STAGES;
          if (n > 0) ok = ptx::mbar_wait(bars + L::KV_EMPTY + s, (n - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          uint8_t* ks = sm + L::KV_OFF + 2 * s * L::TILE;
          ptx::mbar_expect_tx(bars + L::K_FULL + s, L::TILE);
          load_key_tile<DT>(&maps.k, ks, w.b, w.hk, w.t0 + t, p.s.k_b, p.s.k_h, bars + L::K_FULL + s);
          ptx::mbar_expect_tx(bars + L::V_FULL + s, L::TILE);
          load_key_tile<DT>(&maps.v, ks + L::TILE, w.b, w.hk, w.t0 + t, p.s.v_b, p.s.v_h, bars + L::V_FULL + s);
        }
      }
      // drain: every issued load has landed before the CTA may exit
      for (int x = 0; x < 2; ++x)
        if (nqx[x] > 0) ptx::mbar_drain(bars + L::Q_FULL + x, (nqx[x] - 1) & 1, 100000000ll);
      for (int k = max(0, kv - L::STAGES); k < kv; ++k) {
        ptx::mbar_drain(bars + L::K_FULL + k % L::STAGES, (k / L::STAGES) & 1, 100000000ll);
        ptx::mbar_drain(bars + L::V_FULL + k % L::STAGES, (k / L::STAGES) & 1, 100000000ll);
      }
    } else if (warp == 1 && lane == 0) {
      // ====================================== MMA issuer ======================================
      // In each unit ns[x] and np[x] are the next S and P V of tile x. The loop polls and issues
      // what is ready, each tile's P V before either S: the pipe runs products in issue order,
      // and a P V gates its tile's next S and the key tile's release.
      const uint32_t sQ = ptx::smem_u32(sm + L::Q_OFF), sKV = ptx::smem_u32(sm + L::KV_OFF);
      const uint32_t id_o = ptx::idesc_bf16(128, dsteps * 16, 0, 1);
      constexpr uint32_t TILE16 = L::TILE >> 4, MN_STEP = 2048 >> 4;
      FwdWalk w(p);
      int tq[2] = {0, 0}, ts[2] = {0, 0}, tp[2] = {0, 0};   // units, S and P V of tile x so far
      int kv0 = 0;
      uint32_t clean = 0;                          // parities of the stages' CLEAN barriers
      bool ok = true;
      long long t_last = global_timer_ns();
      while (ok && w.next()) {
        if (w.nt == 0) continue;
        const int ntx[2] = {w.nt, w.has_b ? w.nt : 0};
        const int dirty = w.unclean(w.nt - 1) ? w.nt - 1 : -1;   // the last tile alone can be
        int ns[2] = {0, 0}, np[2] = {0, 0}, released = 0;
        while (ok && (np[0] < ntx[0] || np[1] < ntx[1])) {
          bool progress = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = np[x], s = (kv0 + t) % L::STAGES;
            if (t < ns[x] && mbar_test(bars + L::P_FULL + x, tp[x] & 1) &&
                mbar_test(bars + L::V_FULL + s, ((kv0 + t) / L::STAGES) & 1) &&
                (t != dirty || mbar_test(bars + L::CLEAN + s, (clean >> s) & 1))) {
              ptx::tc_fence_after();
              const uint32_t dV = ptx::sdesc_lo(sKV + (2 * s + 1) * L::TILE, kTile * 128);
              const int steps = 2 * w.chunks(t);
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                if (ks < steps)
                  ptx::mma_ts(tmem + L::T_O + DT * x, tmem + L::T_P + L::P_STRIDE * x + 8 * ks, dV + ks * MN_STEP,
                              id_o, (t > 0 || ks > 0) ? 1u : 0u);
              ptx::mma_commit(bars + L::PV_DONE + x);
              ++np[x];
              ++tp[x];
              progress = true;
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = ns[x], s = (kv0 + t) % L::STAGES;
            // S_x follows the tile's last P V (over whose P it is written when DT = 128)
            if (t < ntx[x] && t == np[x] && mbar_test(bars + L::K_FULL + s, ((kv0 + t) / L::STAGES) & 1) &&
                (t > 0 || mbar_test(bars + L::Q_FULL + x, tq[x] & 1)) &&
                (L::kSepP || tp[x] == 0 || mbar_test(bars + L::PV_DONE + x, (tp[x] - 1) & 1))) {
              ptx::tc_fence_after();
              const uint32_t id_s = ptx::idesc_bf16(128, 32 * w.chunks(t), 0, 0);
              const uint32_t dQ = ptx::sdesc_lo(sQ, 16) + x * TILE16;
              const uint32_t dK = ptx::sdesc_lo(sKV, 16) + 2 * s * TILE16;
#pragma unroll
              for (int ks = 0; ks < DT / 16; ++ks) {
                const uint32_t step = ((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4;
                if (ks < dsteps) ptx::mma_lo(tmem + L::T_S + 128 * x, dQ + step, dK + step, id_s, ks > 0);
              }
              ptx::mma_commit(bars + L::S_FULL + x);
              if (t == w.nt - 1) {
                ptx::mma_commit(bars + L::Q_EMPTY + x);
                ++tq[x];
              }
              ++ns[x];
              ++ts[x];
              progress = true;
            }
          }
          while (released < w.nt && np[0] > released && (!w.has_b || np[1] > released)) {
            ptx::mma_commit(bars + L::KV_EMPTY + (kv0 + released) % L::STAGES);
            ++released;
          }
          if (progress) {
            t_last = global_timer_ns();
          } else if (*abort_flag) {
            ok = false;
          } else if (global_timer_ns() - t_last > tmo) {
            *abort_flag = 1;
            ok = false;
          }
        }
        if (dirty >= 0) clean ^= 1u << ((kv0 + dirty) % L::STAGES);
        kv0 += w.nt;
      }
      ptx::mma_commit(bars + L::DRAIN);
      ptx::mbar_drain(bars + L::DRAIN, 0, 1000000000ll);
    } else if (warp == 2 && p.s.lens) {
      // ============================ rows of V behind a sequence's end ==========================
      // Every tile is waited for and its stage released here too, so that this warp can be neither
      // ahead of the copies nor behind the products by more than a barrier's phase.
      FwdWalk w(p);
      int kv = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int t = 0; t < w.nt; ++t, ++kv) {
          const int s = kv % L::STAGES;
          ok = ptx::warp_wait(bars + L::V_FULL + s, (kv / L::STAGES) & 1, abort_flag, tmo);
          if (!ok) break;
          if (t == w.nt - 1 && w.unclean(t)) {
            clear_rows<DT>(sm + L::KV_OFF + (2 * s + 1) * L::TILE, w.keys(t), 32 * w.chunks(t), lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bars + L::CLEAN + s);
          }
          if (lane == 0) ptx::mbar_arrive(bars + L::KV_EMPTY + s);
        }
      }
    }
  } else {
    ptx::regs_inc<kFwdRegsSoftmax>();
    // ======================================= softmax ========================================
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;             // row within the tile = TMEM lane
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = tmem + lane_addr + L::T_S + 128 * x;
    const uint32_t t_pp = tmem + lane_addr + L::T_P + L::P_STRIDE * x;
    const uint32_t t_o = tmem + lane_addr + L::T_O + DT * x;
    FwdWalk w(p);
    int steps = 0;                                 // key tiles so far: parity of this tile's barriers
    bool ok = true;
    while (w.next()) {
      if (x && !w.has_b) continue;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; ok && t < w.nt; ++t) {
        ok = ptx::warp_wait(bars + L::S_FULL + x, steps & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        const int keys = w.keys(t), chunks = (keys + 31) >> 5;
        uint32_t sc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) ptx::tmem_ld32_issue(t_s + 32 * c, sc[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) ptx::tmem_ld32_wait(sc[c]);
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < chunks) {
            if (32 * c + 32 > keys) {              // the sequence ends in this chunk
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= keys) sc[c][i] = 0xff800000u;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], __uint_as_float(sc[c][i]), __uint_as_float(sc[c][i + 1]));
          }
        }
        const float m_row = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
        const bool moved = m_row > m + kRescaleLog2;
        const float m_new = moved ? m_row : m;
        const uint64_t scale2 = two(p.scale_log2, p.scale_log2), off2 = two(-m_new, -m_new);
        uint64_t lt[2] = {0ull, 0ull};             // four partial sums
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < chunks) {
            uint32_t u[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float e0, e1;
              exp2_two(__uint_as_float(sc[c][2 * k]), __uint_as_float(sc[c][2 * k + 1]), scale2, off2, e0, e1);
              lt[k & 1] = add2(lt[k & 1], two(e0, e1));
              u[k] = ptx::pack_bf16(e0, e1);
            }
            ptx::tmem_st8(t_pp + 16 * c, u);
            ptx::tmem_st8(t_pp + 16 * c + 8, u + 8);
          }
        }
        float lt0, lt1;
        untwo(add2(lt[0], lt[1]), lt0, lt1);
        const float alpha = moved ? ptx::ex2(m - m_new) : 1.f;
        l = l * alpha + (lt0 + lt1);
        m = m_new;
        // the products before this S have ended, O's last one among them
        if (t > 0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int c0 = 0; c0 < DT; c0 += 32) {
            if (c0 < p.s.D) {
              uint32_t a[32];
              ptx::tmem_ld32_issue(t_o + c0, a);
              ptx::tmem_ld32_wait(a);
#pragma unroll
              for (int c = 0; c < 32; ++c) a[c] = __float_as_uint(__uint_as_float(a[c]) * alpha);
              ptx::tmem_st32(t_o + c0, a);
            }
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + L::P_FULL + x);
        ++steps;
      }
      if (ok && w.nt > 0) ok = ptx::warp_wait(bars + L::PV_DONE + x, (steps - 1) & 1, abort_flag, tmo);
      if (ok) ptx::tc_fence_after();
      int token, head;
      const int tile = 2 * w.pair + x;
      const bool live = row_of(p.s, tile, r, token, head);
      const bool none = w.nt == 0;                 // no key: O = 0, LSE = -inf (NaN for a bad length)
      const bool bad = !ok || w.len < 0;
      const float inv = bad ? NAN : none ? 0.f : 1.f / l;
      const float l2 = bad ? NAN : none ? -INFINITY : m + __log2f(l);
      if (p.splits > 1) {
        const size_t row = (((size_t)w.split * p.s.B * p.s.Hk + w.bh) * p.s.ntile + tile) * kTile + r;
        if (live) p.part_l[row] = l2;
        if (!none && ok) {
#pragma unroll
          for (int c0 = 0; c0 < DT; c0 += 32) {
            if (c0 < p.s.D) {
              float v[32];
              ptx::tmem_ld32(t_o + c0, v);
              if (live) {
                float4* d4 = (float4*)(p.part_o + row * DT + c0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  d4[k] = make_float4(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
              }
            }
          }
        }
      } else {
        const int h = w.hk * p.s.g + head;
        if (live) p.lse[((size_t)w.b * p.s.Hq + h) * p.s.Sq + token] = l2 * kLn2;
        __nv_bfloat16* dst = p.o + (((size_t)w.b * p.s.Sq + token) * p.s.Hq + h) * p.s.D;
#pragma unroll
        for (int c0 = 0; c0 < DT; c0 += 32) {
          if (c0 < p.s.D) {
            float v[32];
            if (none || bad) {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = 1.f;
            } else {
              ptx::tmem_ld32(t_o + c0, v);
            }
            if (live) store_bf16_32(dst + c0, v, inv, p.s.D - c0);
          }
        }
      }
      // O has been read: the next unit's P V may replace it, which waits for this warp's P
      ptx::tc_fence_before();
      if (w.len < 0 && w.pair == 0 && x == 0 && r == 0 && p.status) atomicCAS(p.status, 0, kStatusBounds);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag && p.status) atomicCAS(p.status, 0, kStatusSyncTimeout);
}

// The ranges of keys of one row, combined in order: O = sum 2^(l_s - M) O_s / sum 2^(l_s - M). A
// warp a row; ranges without keys have l_s = -inf and nothing in part_o.
template <int DT>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ FwdArgs p) {
  constexpr int PER = DT / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.s.B * p.s.Hk * p.s.ntile * kTile;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  train::grid_wait();
  if (row >= rows) return;
  const int r = (int)(row % kTile);
  const long long rest = row / kTile;
  const int tile = (int)(rest % p.s.ntile), bh = (int)(rest / p.s.ntile);
  const int b = bh / p.s.Hk, hk = bh - b * p.s.Hk;
  int token, head;
  if (!row_of(p.s, tile, r, token, head)) return;
  float mx = -INFINITY;
  bool nan = false;
  for (int s = lane; s < p.splits; s += 32) {
    const float l2 = p.part_l[s * rows + row];
    nan |= isnan(l2);
    mx = fmaxf(mx, l2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  nan = __any_sync(0xffffffffu, nan);
  float acc[PER] = {}, total = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float l2 = p.part_l[s * rows + row];
    if (!(l2 > -INFINITY)) continue;
    const float f = ptx::ex2(l2 - mx);
    total += f;
    const float* src = p.part_o + ((size_t)s * rows + row) * DT + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = fmaf(f, src[i], acc[i]);
  }
  const float inv = nan ? NAN : total > 0.f ? 1.f / total : 0.f;
  const int h = hk * p.s.g + head;
  if (lane == 0)
    p.lse[((size_t)b * p.s.Hq + h) * p.s.Sq + token] =
        nan ? NAN : total > 0.f ? (mx + __log2f(total)) * kLn2 : -INFINITY;
  if (lane * PER < p.s.D) {
    __nv_bfloat16* dst = p.o + (((size_t)b * p.s.Sq + token) * p.s.Hq + h) * p.s.D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; i += 2)
      *reinterpret_cast<uint32_t*>(dst + i) = ptx::pack_bf16(acc[i] * inv, acc[i + 1] * inv);
  }
}

}  // namespace cross
}  // namespace dash
