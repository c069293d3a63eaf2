// Cross attention forward: O = softmax(scale Q K^T over the batch's keys) V and the natural-log
// LSE per row, on the 5th-generation tensor cores.
//
// A unit of work is a pair of row tiles (A and B) of one group of heads and a range of key tiles;
// a persistent grid runs the units in turn. Each row tile has eight softmax warps, an issuer and
// TMEM of its own, both walk the same key tiles:
//   S_x = Q_x K_j^T       M = 128 rows, N = the tile's keys, K = D      TMEM cols [128 x, +128)
//   P_x = exp2(S_x scale log2e - m)      packed bf16: over S_x's first 64 columns (DT = 128) or in
//                                        64 columns of its own (DT = 64)
//   O_x += P_x V_j        M = 128, N = D, K = the tile's keys           TMEM cols [256 + DT x, +DT)
// While one tile's warps turn S into P the products of the other run, and while a unit's rows leave
// for memory the next unit's tiles load and its first S is computed. The last key tile of a
// sequence takes only its 32-column chunks with keys (77 keys: 96 columns, not 128).
// A softmax thread owns half a row: it takes its scores out of TMEM once, so the maximum and the
// exponentials need no second read, and moves the exponent's reference m only when the row
// maximum exceeds it by more than 8 in log2 units (P <= 2^8; O and l share the reference).
//
// Bound, with long states, by the tensor cores and the turns: of a tile's 1750 cycles 1024 are
// products, the rest the ways from P to its issuer, from O to S and to the other tile. 8192 x 8192 x 128,
// 32 heads, takes 773 to 832 us (1322 to 1422 TFLOP/s by card), 4096 x 4096 x 64, 32 heads, where the
// products have half the work for the same softmax, 195 to 213. With captions a unit is one step and its
// ends: 16 heads of 64, 4 x 4096 rows x 77 keys, 27 us where the bytes take 10.
//
// Key ranges (splits > 1): where the pairs of row tiles would leave most of the chip idle (single
// tokens against long states) the keys are cut into ranges; a range leaves its rows' normalised O
// in fp32 and their LSE, which cross_join_kernel combines in order.
//
// Warp roles (640 threads): 0 = TMA producer, 1 and 3 = MMA issuers of tiles A and B, 2 = clears V
// rows that a length leaves out, 4..11 = softmax of tile A, 12..19 = of tile B. Every wait is
// bounded; a CTA that gives up writes NaN into the LSE of its rows and records
// DASH_ERR_SYNC_TIMEOUT where asked to.
#pragma once

#include "cross_common.cuh"

namespace dash {
namespace cross {

struct FwdArgs {
  Shape s;
  __nv_bfloat16* o;          // [B, Sq, Hq, D]
  float* lse;                // [B, Hq, Sq]
  float* part_o;             // splits > 1: [split][group][tile][DT / 8][128][8]
  float* part_l;             //             [split][group][tile][128] LSE in log2 units
  int pairs, splits, kper;   // pairs of row tiles a group; key ranges, key tiles a range
  Units units;
  float scale_log2;
  int* status;
  long long timeout_ns;
  int withhold;              // testing hook: load no keys, so that the waits for them run out
};

template <int DT>
struct FwdLay {
  static constexpr int TILE = kTile * DT * 2;
  static constexpr int KST = DT == 64 ? 4 : 2, VST = DT == 64 ? 4 : 3;   // stages of K and V
  static constexpr int Q_OFF = 0, K_OFF = 2 * TILE, V_OFF = K_OFF + KST * TILE;
  static constexpr int EX_OFF = V_OFF + VST * TILE;           // the halves of a row: [tile][half][128]
  static constexpr int BAR_OFF = EX_OFF + 4 * kTile * 4;
  static constexpr int ALLOC = BAR_OFF + 512;                 // the base is 1024-aligned (checked)
  static_assert(ALLOC <= 232448, "shared memory budget");
  static constexpr int T_S = 0, T_O = 256;
  static constexpr bool kSepP = DT == 64;                     // P in columns of its own
  static constexpr int T_P = kSepP ? T_O + 2 * DT : T_S;
  static constexpr int P_STRIDE = kSepP ? 64 : 128;
  static_assert(T_O + 2 * DT + (kSepP ? 128 : 0) <= 512, "TMEM columns");
  // barriers
  static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 6, PV_DONE = 8, DRAIN = 10, TURN = 12,
                       K_FULL = 14, V_FULL = K_FULL + KST, K_EMPTY = V_FULL + VST, V_EMPTY = K_EMPTY + KST,
                       CLEAN = V_EMPTY + VST, COUNT = CLEAN + VST;
  static_assert(8 * COUNT + 8 <= 512, "barrier area");
};

constexpr int kFwdThreads = 640;
constexpr float kRescaleLog2 = 8.f;
// The reference of a row without a score above -inf so far: finite, so that such scores get the weight
// exp2(-inf) = 0 (around a reference of -inf it would be NaN) and a later one moves it.
constexpr float kLowest = -3.4028234663852886e38f;
constexpr int kFwdRegsLaunch = 96, kFwdRegsCtrl = 32, kFwdRegsSoftmax = 112;
static_assert(kFwdRegsCtrl + 4 * kFwdRegsSoftmax == 5 * kFwdRegsLaunch,
              "the five warpgroups must share exactly the launch's registers");

// A CTA's units, [batch][pair][key head][split]. Every role walks the same ones. ALL: a whole warp
// walks together.
template <bool ALL = false>
struct FwdWalk {
  const FwdArgs* a;
  Place at;                  // d0: key range, d1: pair of row tiles
  int known;                 // the batch whose length is at hand (-2: not begun)
  int len;                   // the batch's keys (-1: out of range)
  int t0, nt;                // first key tile and their number in this range
  bool has_b;
  __device__ __forceinline__ FwdWalk(const FwdArgs& args) : a(&args), at(args.units), known(-2) {}
  __device__ __forceinline__ bool next() {
    const FwdArgs& p = *a;
    if (known == -2) known = -1;
    else at.next(p.units);
    if (!at.more(p.units)) return false;
    has_b = 2 * at.d1 + 1 < p.s.ntile;
    if (at.b != known) {
      known = at.b;
      len = length_of(p.s, known);
      if (ALL) len = same(len);
    }
    t0 = at.d0 * p.kper;
    const int all = (max(len, 0) + kTile - 1) / kTile;
    nt = max(0, min(all, t0 + p.kper) - t0);
    return true;
  }
  // The keys of a place's range (none: 0 or less).
  __device__ static __forceinline__ int keys_in_range(const FwdArgs& p, const Place& at) {
    return min(length_of(p.s, at.b) - at.d0 * p.kper * kTile, p.kper * kTile);
  }
  __device__ __forceinline__ int group() const { return at.b * a->s.Hk + at.hk; }
  // Keys of key tile t of this range, and how many 32-column chunks they take.
  __device__ __forceinline__ int keys(int t) const { return min(kTile, len - (t0 + t) * kTile); }
  __device__ __forceinline__ int chunks(int t) const { return (keys(t) + 31) >> 5; }
  // Rows of the V tile that the product reads although the length leaves them out (rows beyond
  // the tensor arrive as zeros).
  __device__ __forceinline__ bool unclean(int t) const { return len < a->s.Sk && (keys(t) & 31); }
};

template <int DT>
__global__ void __launch_bounds__(kFwdThreads, 1)
    cross_fwd_kernel(const __grid_constant__ FwdArgs p, const __grid_constant__ Maps maps) {
  using L = FwdLay<DT>;
  extern __shared__ __align__(1024) uint8_t smem_cross[];
  uint8_t* sm = smem_cross;
  uint64_t* bars = (uint64_t*)(sm + L::BAR_OFF);
  uint32_t* tmem_slot = (uint32_t*)(sm + L::BAR_OFF + 8 * L::COUNT);
  volatile int* abort_flag = (volatile int*)(sm + L::BAR_OFF + 8 * L::COUNT + 4);
  const int warp = same((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const long long tmo = p.timeout_ns;
  const int dsteps = (p.s.D + 15) >> 4;

  if (p.splits > 1) train::grid_next();
  // The layout fills most of the opt-in maximum, so there is no room to realign the base.
  if (ptx::smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, kStatusSmemLayout);
    return;
  }
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
      ptx::mbar_init(bars + L::P_FULL + x, 8);
      ptx::mbar_init(bars + L::PV_DONE + x, 1);
    }
    for (int s = 0; s < L::KST; ++s) {
      ptx::mbar_init(bars + L::K_FULL + s, 1);
      ptx::mbar_init(bars + L::K_EMPTY + s, 2);                   // both tiles
    }
    for (int s = 0; s < L::VST; ++s) {
      ptx::mbar_init(bars + L::V_FULL + s, 1);
      ptx::mbar_init(bars + L::V_EMPTY + s, p.s.lens ? 3 : 2);   // and warp 2
      ptx::mbar_init(bars + L::CLEAN + s, 1);
    }
    ptx::mbar_init(bars + L::DRAIN, 1);
    ptx::mbar_init(bars + L::DRAIN + 1, 1);
    ptx::mbar_init(bars + L::TURN, 1);
    ptx::mbar_init(bars + L::TURN + 1, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);

  if (warp < 4) {
    ptx::regs_dec<kFwdRegsCtrl>();
    if (warp == 0 && lane == 0) {
      // ===================================== TMA producer =====================================
      FwdWalk<> w(p);
      int nqx[2] = {0, 0}, nk = 0, nv = 0;         // row tiles, tiles of K and V loaded so far
      bool ok = true;
      while (ok && w.next()) {
        if (w.nt == 0) continue;
        for (int x = 0; ok && x < (w.has_b ? 2 : 1); ++x) {
          if (nqx[x] > 0) ok = ptx::mbar_wait(bars + L::Q_EMPTY + x, (nqx[x] - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::Q_FULL + x, row_tile_bytes<DT>(p.s));
          load_row_tile<DT>(p.s, &maps.q, sm + L::Q_OFF + x * L::TILE, w.at.b, w.at.hk, 2 * w.at.d1 + x, p.s.q_b, p.s.q_h,
                            bars + L::Q_FULL + x);
          ++nqx[x];
        }
        for (int t = 0; ok && t < (p.withhold ? 0 : w.nt); ++t) {
          const int ks = nk % L::KST, km = nk / L::KST, vs = nv % L::VST, vm = nv / L::VST;
          if (km > 0) ok = ptx::mbar_wait(bars + L::K_EMPTY + ks, (km - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::K_FULL + ks, L::TILE);
          load_key_tile<DT>(&maps.k, sm + L::K_OFF + ks * L::TILE, w.at.b, w.at.hk, w.t0 + t, p.s.k_b, p.s.k_h,
                            bars + L::K_FULL + ks);
          ++nk;
          if (vm > 0) ok = ptx::mbar_wait(bars + L::V_EMPTY + vs, (vm - 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::mbar_expect_tx(bars + L::V_FULL + vs, L::TILE);
          load_key_tile<DT>(&maps.v, sm + L::V_OFF + vs * L::TILE, w.at.b, w.at.hk, w.t0 + t, p.s.v_b, p.s.v_h,
                            bars + L::V_FULL + vs);
          ++nv;
        }
      }
      // drain: every issued load has landed before the CTA may exit
      for (int x = 0; x < 2; ++x)
        if (nqx[x] > 0) ptx::mbar_drain(bars + L::Q_FULL + x, (nqx[x] - 1) & 1, 100000000ll);
      for (int k = max(0, nk - L::KST); k < nk; ++k)
        ptx::mbar_drain(bars + L::K_FULL + k % L::KST, (k / L::KST) & 1, 100000000ll);
      for (int k = max(0, nv - L::VST); k < nv; ++k)
        ptx::mbar_drain(bars + L::V_FULL + k % L::VST, (k / L::VST) & 1, 100000000ll);
    } else if (warp == 1 || warp == 3) {
      // ================================ MMA issuer of tile x ==================================
      // S(t) needs K(t); over P's columns (DT = 128) also P(t-1) V(t-1) done. With P in columns of
      // its own (DT = 64) S(t+1) goes ahead of P(t) V(t).
      // Over several key tiles the two issuers take turns with P(t) V(t) and S(t+1), so that one
      // tile's products run while the other's scores become P. Left alone they fall into step, both
      // in the softmax and then both in line for the pipe (8192 x 8192 x 128, 32 heads, when this was built:
      // 1237 us, with turns 1092; a turn that passes before S is all issued: 829 for 806). With one or two
      // key tiles turns only cost (77 keys: 33 us, with turns 38).
      const int x = warp >> 1;
      const uint32_t dQ = ptx::sdesc_lo(ptx::smem_u32(sm + L::Q_OFF + x * L::TILE), 16);
      const uint32_t sK = ptx::smem_u32(sm + L::K_OFF), sV = ptx::smem_u32(sm + L::V_OFF);
      const uint32_t id_o = ptx::idesc_bf16(128, dsteps * 16, 0, 1);
      FwdWalk<true> w(p);
      const uint32_t one = elect_one();
      int n = 0, k = 0, pv = 0, turns = 0;         // this tile's units, products P V and turns, all key tiles so far
      uint32_t clean = 0;                          // parities of the stages' CLEAN barriers
      bool ok = true;
      while (ok && w.next()) {
        if (w.nt == 0) continue;
        const bool last_dirty = w.unclean(w.nt - 1);
        if (x && !w.has_b) {                       // nothing to issue: the stages are released all the same
          for (int t = 0; ok && t < w.nt; ++t) {
            const int ks = (k + t) % L::KST, vs = (k + t) % L::VST;
            ok = ptx::warp_wait(bars + L::K_FULL + ks, ((k + t) / L::KST) & 1, abort_flag, tmo);
            if (ok && one) ptx::mbar_arrive(bars + L::K_EMPTY + ks);
            if (ok) ok = ptx::warp_wait(bars + L::V_FULL + vs, ((k + t) / L::VST) & 1, abort_flag, tmo);
            if (ok && t == w.nt - 1 && last_dirty) {
              ok = ptx::warp_wait(bars + L::CLEAN + vs, (clean >> vs) & 1, abort_flag, tmo);
              clean ^= 1u << vs;
            }
            if (ok && one) ptx::mbar_arrive(bars + L::V_EMPTY + vs);
          }
          k += w.nt;
          continue;
        }
        const bool take_turns = w.has_b && w.nt > 2;
        auto issue_s = [&](int t, bool landed) {
          const int s = (k + t) % L::KST;
          bool good = landed || ptx::warp_wait(bars + L::K_FULL + s, ((k + t) / L::KST) & 1, abort_flag, tmo);
          if (good && !L::kSepP && pv > 0) good = ptx::warp_wait(bars + L::PV_DONE + x, (pv - 1) & 1, abort_flag, tmo);
          if (!good) return false;
          ptx::tc_fence_after();
          const uint32_t id_s = ptx::idesc_bf16(128, 32 * w.chunks(t), 0, 0);
          const uint32_t dK = ptx::sdesc_lo(sK + s * L::TILE, 16);
          issue_scores<DT>(tmem + L::T_S + 128 * x, dQ, dK, id_s, dsteps, one);
          commit(bars + L::S_FULL + x, one);
          commit(bars + L::K_EMPTY + s, one);
          if (t == w.nt - 1) commit(bars + L::Q_EMPTY + x, one);
          return true;
        };
        ok = ptx::warp_wait(bars + L::Q_FULL + x, n & 1, abort_flag, tmo) && issue_s(0, false);
        for (int t = 0; ok && t < w.nt; ++t) {
          const int s = (k + t) % L::VST, nk = k + t + 1, ns = nk % L::KST;
          // what else the products wait for comes before P and the turn, out of the way (a wait costs 100
          // cycles when it is over already; all of them in the way: 880 us in place of 782 at 16384 x 4096)
          ok = ptx::warp_wait(bars + L::V_FULL + s, ((k + t) / L::VST) & 1, abort_flag, tmo);
          if (ok && t == w.nt - 1 && last_dirty) {
            ok = ptx::warp_wait(bars + L::CLEAN + s, (clean >> s) & 1, abort_flag, tmo);
            clean ^= 1u << s;
          }
          const bool landed = t + 1 < w.nt && is_complete(bars + L::K_FULL + ns, (nk / L::KST) & 1);
          // A's first turn ever is its own; A's turn n waits for B's turn n - 1, B's for A's turn n
          if (ok && take_turns && (x || turns > 0))
            ok = ptx::warp_wait(bars + L::TURN + x, (x ? turns : turns - 1) & 1, abort_flag, tmo);
          if (ok) ok = ptx::warp_wait(bars + L::P_FULL + x, pv & 1, abort_flag, tmo);
          if (ok && L::kSepP && t + 1 < w.nt) ok = issue_s(t + 1, landed);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t dV = ptx::sdesc_lo(sV + s * L::TILE, kTile * 128);
          issue_rows<false>(tmem + L::T_O + DT * x, tmem + L::T_P + L::P_STRIDE * x, dV, id_o, t > 0 ? 1u : 0u,
                            2 * w.chunks(t), one);
          commit(bars + L::PV_DONE + x, one);
          commit(bars + L::V_EMPTY + s, one);
          ++pv;
          if (!L::kSepP && t + 1 < w.nt) ok = issue_s(t + 1, landed);
          if (take_turns) {
            ++turns;
            if (one) ptx::mbar_arrive(bars + L::TURN + 1 - x);
          }
        }
        k += w.nt;
        ++n;
      }
      commit(bars + L::DRAIN + x, one);
      ptx::mbar_drain(bars + L::DRAIN + x, 0, 1000000000ll);
    } else if (warp == 2 && p.s.lens) {
      // ============================ rows of V behind a sequence's end ==========================
      // Every tile is waited for and its stage released here too, so that this warp can be neither
      // ahead of the copies nor behind the products by more than a barrier's phase.
      FwdWalk<> w(p);
      int kv = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int t = 0; t < w.nt; ++t, ++kv) {
          const int s = kv % L::VST;
          ok = ptx::warp_wait(bars + L::V_FULL + s, (kv / L::VST) & 1, abort_flag, tmo);
          if (!ok) break;
          if (t == w.nt - 1 && w.unclean(t)) {
            clear_rows<DT>(sm + L::V_OFF + s * L::TILE, w.keys(t), 32 * w.chunks(t), lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bars + L::CLEAN + s);
          }
          if (lane == 0) ptx::mbar_arrive(bars + L::V_EMPTY + s);
        }
      }
    }
  } else {
    ptx::regs_inc<kFwdRegsSoftmax>();
    // ======================================= softmax ========================================
    // Two warps a quarter of a tile: a thread owns a row's 64 keys of its half, and of O its half of
    // the columns. The halves share the row's maximum and sum through shared memory.
    const int x = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;             // row within the tile = TMEM lane
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = tmem + lane_addr + L::T_S + 128 * x + 64 * half;
    const uint32_t t_pp = tmem + lane_addr + L::T_P + L::P_STRIDE * x + 32 * half;
    const uint32_t t_o = tmem + lane_addr + L::T_O + DT * x;
    float* mine = (float*)(sm + L::EX_OFF) + (x * 2 + half) * kTile + r;
    const float* other = (const float*)(sm + L::EX_OFF) + (x * 2 + 1 - half) * kTile + r;
    const int pair_bar = 1 + x * 4 + quarter;      // the two warps' named barrier
    // (Registers are short here, and a spilled one costs more than a length read again: of the walk
    // only the place is kept, and of its keys how many are left.)
    Place at(p.units);
    int steps = 0;                                 // key tiles so far: parity of this tile's barriers
    bool ok = true;
    for (; at.more(p.units); at.next(p.units)) {
      if (x && 2 * at.d1 + 1 >= p.s.ntile) continue;
      float m = kLowest, l = 0.f;                  // of the row; of this half
      bool first = true;                           // key tile of the unit
      // A warp whose wait ran out goes on without work, as its partner must find it at every meeting.
      for (int left = FwdWalk<>::keys_in_range(p, at); left > 0; left -= kTile, ++steps) {
        if (ok) ok = ptx::warp_wait(bars + L::S_FULL + x, steps & 1, abort_flag, tmo);
        ptx::tc_fence_after();
        const int keys = min(left, kTile) - 64 * half;   // of this half
        uint32_t sc[2][32];
        float mx = -INFINITY;
        if (ok) {
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (32 * c < keys) ptx::tmem_ld32_issue(t_s + 32 * c, sc[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (32 * c < keys) ptx::tmem_ld32_wait(sc[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (32 * c < keys) {
              if (32 * c + 32 > keys) {            // the sequence ends in this chunk
                const uint32_t there = (1u << (keys - 32 * c)) - 1u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(there >> i & 1u)) sc[c][i] = 0xff800000u;
              }
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], __uint_as_float(sc[c][i]), __uint_as_float(sc[c][i + 1]));
            }
          }
          mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
        }
        // The place is the partner's to read until its P is stored, which the next S waits for. The
        // meeting also says that both halves' scores have been read: P lies over half 0's (DT = 128).
        *mine = mx;
        ptx::tc_fence_before();
        ptx::named_bar(pair_bar, 64);
        ptx::tc_fence_after();
        if (!ok) continue;
        const float m_row = fmaxf(mx, *other) * p.scale_log2;
        const bool moved = m_row > m + kRescaleLog2;
        const float m_new = moved ? m_row : m;
        // P's columns, and O where it is rescaled, are the last product's until that is done (DT = 128: it
        // was, before this S)
        if (L::kSepP && !first) {
          ok = ptx::warp_wait(bars + L::PV_DONE + x, (steps - 1) & 1, abort_flag, tmo);
          if (!ok) continue;
          ptx::tc_fence_after();
        }
        const uint64_t scale2 = two(p.scale_log2, p.scale_log2), off2 = two(-m_new, -m_new);
        uint64_t lt[2] = {0ull, 0ull};             // four partial sums
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (32 * c < keys) {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
              uint32_t u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float e0, e1;
                exp2_two(__uint_as_float(sc[c][2 * (k + i)]), __uint_as_float(sc[c][2 * (k + i) + 1]), scale2, off2, e0, e1);
                lt[i & 1] = add2(lt[i & 1], two(e0, e1));
                u[i] = ptx::pack_bf16(e0, e1);
              }
              ptx::tmem_st8(t_pp + 16 * c + k, u);
            }
          }
        }
        float lt0, lt1;
        untwo(add2(lt[0], lt[1]), lt0, lt1);
        const float alpha = moved ? ptx::ex2(m - m_new) : 1.f;
        l = l * alpha + (lt0 + lt1);
        m = m_new;
        if (!first && __any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < DT / 2; i += 32) {
            const int c0 = half * (DT / 2) + i;
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
        first = false;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + L::P_FULL + x);
      }
      const int len = length_of(p.s, at.b);
      const bool none = FwdWalk<>::keys_in_range(p, at) <= 0;   // no key: O = 0, LSE = -inf
      if (!none) {
        if (ok) ok = ptx::warp_wait(bars + L::PV_DONE + x, (steps - 1) & 1, abort_flag, tmo);
        ptx::tc_fence_after();
        // the row's sum; the maxima in these places have been read, as above
        *mine = l;
        ptx::named_bar(pair_bar, 64);
        l += *other;
        ptx::named_bar(pair_bar, 64);
      }
      int token, head;
      const int tile = 2 * at.d1 + x, group = at.b * p.s.Hk + at.hk;
      const bool live = row_of(p.s, tile, r, token, head);
      const bool bad = !ok || len < 0;             // NaN for a bad length
      const float inv = bad ? NAN : none || l == 0.f ? 0.f : 1.f / l;   // l = 0: all scores are -inf
      const float l2 = bad ? NAN : none ? -INFINITY : m + __log2f(l);
      const size_t row = (((size_t)at.d0 * p.s.B * p.s.Hk + group) * p.s.ntile + tile) * kTile + r;
      const int h = at.hk * p.s.g + head;
      if (live && half == 0) {
        if (p.splits > 1) p.part_l[row] = l2;
        else p.lse[((size_t)at.b * p.s.Hq + h) * p.s.Sq + token] = l2 * kLn2;
      }
      __nv_bfloat16* dst = p.o + (((size_t)at.b * p.s.Sq + token) * p.s.Hq + h) * p.s.D;
#pragma unroll
      for (int i = 0; i < DT / 2; i += 32) {
        const int c0 = half * (DT / 2) + i;
        if (c0 < p.s.D) {
          float v[32];
          if (none || bad) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = 1.f;
          } else {
            ptx::tmem_ld32(t_o + c0, v);
          }
          if (p.splits == 1) store_rows_bf16(lane, v, inv, live ? dst + c0 : nullptr, p.s.D - c0);
          else if (live && !none && ok) store_part_32(p.part_o + (row - r) * DT, r, c0, v, inv);
        }
      }
      // O has been read: the next unit's P V may replace it, which waits for this warp's P
      ptx::tc_fence_before();
      if (len < 0 && at.d1 == 0 && x == 0 && half == 0 && r == 0 && p.status) atomicCAS(p.status, 0, kStatusBounds);
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
  constexpr int PER = DT / 32;                     // columns a lane
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
    const float* src = p.part_o + ((size_t)s * rows + row - r) * DT + part_at(r, lane * PER & ~7) + (lane * PER & 7);
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
