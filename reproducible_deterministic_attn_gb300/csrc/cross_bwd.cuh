// Cross attention backward: dV = P^T dO, dS = P * (dO V^T - Delta), dQ = scale dS K,
// dK = scale dS^T Q with P = exp(scale Q K^T - LSE) recomputed and Delta = rowsum(dO * O).
//
// cross_keys_kernel: a unit of work is one key tile of a group against a segment of its row tiles;
// a persistent grid takes the units in turn. A task is one 128 x 128 tile of scores, with the keys in
// the TMEM lanes:
//   S^T   = K Q^T              M = 128 keys, N = 128 rows, K = D          TMEM cols [0, 128)
//   P^T   = exp2(S^T scale log2e - LSE log2e)            bf16, TMEM, over S^T's columns
//   dP^T  = V dO^T             M = 128 keys, N = 128 rows, K = D          TMEM cols [128, 256)
//   dS^T  = P^T * (dP^T - Delta)                         bf16, TMEM, over dP^T's columns
//   dV   += P^T dO             M = 128 keys, N = D, K = 128 rows, A from TMEM  [256, +DT)
//   dK   += dS^T Q             M = 128 keys, N = D, K = 128 rows, A from TMEM  [256 + DT, +DT)
// dK and dV stay in TMEM over the unit's row tiles. S(t+1) waits for dV(t) (it overwrites P), dP(t+1)
// for dK(t): two chains, each with an issuer of its own, that only the softmax gradient ties together.
// The softmax warps go through exp(t), dS(t), exp(t+1) and would wait for S(t+1), so dK(t) gets in line
// behind dV(t) and S(t+1) (issued as soon as dS(t) is there: 2550 us, so 2430).
// Units of one key tile leave fp32 partials of dK and dV, which cross_join_keys_kernel adds in order.
// A task takes 2600 cycles, 2048 of them products: from P(t) on, 100 until its issuer sees it, dV 700,
// S 750, the exponentials 950. 8192 x 8192 x 128, 32 heads, both kernels: 2350 to 2490 us by card, 1104 to
// 1168 TFLOP/s. P^T in shared memory, which frees S's columns as soon as they are read, gained nothing:
// shared memory has to carry the operands of the products already.
//
// Where a group has one key tile (up to 128 keys: a caption) the same kernel forms dQ too (DQ), as
// nothing has to be summed over key tiles: dS^T also goes to shared memory, [key][row], and
//   dQ^T  = K^T dS^T           M = 128 (d), N = 128 rows, K = keys
// leaves TMEM as bf16 (dS^T is then held over S^T's columns, as dQ^T takes dP^T's when DT = 128).
// Else cross_rows_kernel (cross_bwd_rows.cuh) forms dQ, recomputing S and P a second time: seven
// products instead of five, but nothing to add across units. Adding each task's dQ^T in fp32 in
// global memory instead (each key tile of a unit's row tiles, by the same thread) was slower: 2 x
// 8192 rows x 512 keys x 16 x 128 took 360 us.
// No CTA waits for another one.
//
// -Delta and -LSE log2e come per row from cross_pre_kernel, with -inf for rows a tile does not have and for
// rows whose scores are all -inf (P = 0 there; in a tile without its last row such scores are set to 0
// first, as a row of zeros against an infinite key is NaN). Keys that a length leaves out: warp 2 zeroes
// their rows of K and V in shared memory, as they may hold anything, and their P is set to 0.
//
// Warp roles (512 threads): 0 = TMA producer, 1 and 3 = MMA issuers, 2 = key rows behind a length,
// 4..11 = softmax gradient (quarter = TMEM lanes = keys, half = 64 rows each), 12..15 = dQ
// read-out and the epilogue of dK and dV. Every wait is bounded.
#pragma once

#include "cross_common.cuh"

namespace dash {
namespace cross {

struct BwdArgs {
  Shape s;
  float* nnl;                // [group][tile][128] -LSE log2e
  float* delta;              // [group][tile][128] -Delta
  const __nv_bfloat16 *o, *dO;
  const float* lse;
  __nv_bfloat16 *dq, *dk, *dv;
  long long dq_b, dq_s, dq_h, dk_b, dk_s, dk_h, dv_b, dv_s, dv_h;
  float* dq_part;            // [key segment][group][tile][DT / 8][128][8]
  float* dkv_part;           // [row segment][group][key tile][dK, dV][DT / 8][128][8]
  int qsegs, qper;           // row segments of cross_keys_kernel, row tiles of one
  int ksegs, kper;           // key segments of cross_rows_kernel, key tiles of one
  Units units;               // of the kernel that is being launched
  float scale, scale_log2;
  int* header;
  long long timeout_ns;
  int withhold;
};

template <int DT, bool DQ>
struct KeysLay {
  static constexpr int TILE = kTile * DT * 2;
  static constexpr int DS_BYTES = DQ ? kTile * kTile * 2 : 0;
  static constexpr int OFFS = 2 * kTile * 4;                   // -LSE log2e and -Delta of a row tile
  static constexpr int NQ = DT == 64 || !DQ ? 3 : 2, NDO = DT == 64 ? 3 : 2;
  static constexpr int K_OFF = 0, V_OFF = TILE, Q_OFF = 2 * TILE;
  static constexpr int DO_OFF = Q_OFF + NQ * TILE;
  static constexpr int DS_OFF = DO_OFF + NDO * TILE;
  // DT = 64: zeros after which K^T is padded to 128 rows, so that dQ^T is an M = 128 product
  static constexpr int ZERO_OFF = DS_OFF + DS_BYTES;
  static constexpr int ZERO_BYTES = DQ && DT == 64 ? TILE : 0;
  static constexpr int OFFS_OFF = ZERO_OFF + ZERO_BYTES;
  static constexpr int BAR_OFF = OFFS_OFF + NDO * OFFS;       // (they come and go with dO)
  static constexpr int ALLOC = BAR_OFF + 256;                  // the base is 1024-aligned (checked)
  static_assert(ALLOC <= 232448, "shared memory budget");
  // DT = 64 leaves columns for dQ^T of its own; DT = 128 puts it where dP^T was
  static constexpr bool kSepDQ = DT == 64;
  static constexpr int T_SP = 0, T_DP = 128, T_DV = 256, T_DK = 256 + DT, T_DQ = kSepDQ ? 384 : T_DP;
  static constexpr int T_DS = DQ ? T_SP + 32 : T_DP;           // base of dS^T's packed columns
  static constexpr int REGS_LAUNCH = 128, REGS_SINGLE = 88, REGS_READOUT = 168;
  static_assert(REGS_SINGLE + 2 * REGS_LAUNCH + REGS_READOUT == 4 * REGS_LAUNCH,
                "the four warpgroups must share exactly the launch's registers");
};

enum {
  C_KV_FULL = 0, C_KV_READY, C_KV_EMPTY, C_Q_FULL, C_Q_EMPTY = C_Q_FULL + 3, C_DO_FULL = C_Q_EMPTY + 3,
  C_DO_EMPTY = C_DO_FULL + 3, C_S_FULL = C_DO_EMPTY + 3, C_SP_FREE, C_DP_FREE, C_P_FULL, C_DP_FULL, C_DS_FULL,
  C_DQ_FULL, C_DQ_EMPTY, C_ACC_FULL, C_ACC_EMPTY, C_TURN, C_DRAIN = C_TURN + 2, C_COUNT = C_DRAIN + 2
};
static_assert(8 * C_COUNT + 8 <= 256, "barrier area");

// A CTA's tasks: of each of its units, [batch][row segment][key head][key tile], the row tiles. ALL: a
// whole warp walks together.
template <bool ALL = false>
struct KeysWalk {
  const BwdArgs& p;
  Place at;                  // d0: key tile, d1: row segment
  int known, len;            // the batch whose length is at hand (-2: not begun), that length
  int q0, nqt, j;            // the segment's first row tile, their number, the one at hand
  __device__ __forceinline__ KeysWalk(const BwdArgs& a)
      : p(a), at(a.units), known(-2), len(0), nqt(0), j(0) {}
  __device__ __forceinline__ bool next() {
    if (++j < nqt) return true;
    j = 0;
    do {
      if (known == -2) known = -1;
      else at.next(p.units);
      if (!at.more(p.units)) return false;
      if (at.b != known) {
        known = at.b;
        len = length_of(p.s, known);
        if (ALL) len = same(len);
      }
    } while (at.d0 * kTile >= len);
    q0 = at.d1 * p.qper;
    nqt = min(p.qper, p.s.ntile - q0);
    return true;
  }
  __device__ __forceinline__ int group() const { return at.b * p.s.Hk + at.hk; }
  __device__ __forceinline__ int keys() const { return min(kTile, len - at.d0 * kTile); }
  __device__ __forceinline__ bool first_of_tile() const { return j == 0; }
  __device__ __forceinline__ bool last_of_tile() const { return j == nqt - 1; }
  __device__ __forceinline__ int tile() const { return q0 + j; }
};

// -Delta = -rowsum(dO * O) and -LSE log2e per row; 16 lanes a row, kPreRows rows one after the
// other, in the order in which they lie in memory. Few rows a thread and many threads, as a block
// waits for its loads only once (4 rows and half the threads: 36 us for 134 MB, now 28). Rows of
// batches without keys get their dq here: 0, or NaN for a length out of range. The first block
// clears the workspace's header and looks for such lengths. The next `pads` blocks write the row
// tiles' places that have no row, those behind them dk and dv of the keys that a length leaves out, all of
// them, as a unit's sums for such a key are not zeros where dO is not finite (0 times NaN).
constexpr int kPreRows = 2;
__global__ void __launch_bounds__(256, 8) cross_pre_kernel(const __grid_constant__ BwdArgs p, unsigned row_blocks,
                                                           unsigned pads) {
  train::grid_next();
  if (blockIdx.x == 0) {
    if (threadIdx.x < kWsHeaderBytes / 4) p.header[threadIdx.x] = 0;
    __syncthreads();
    if (p.s.lens)
      for (int b = threadIdx.x; b < p.s.B; b += blockDim.x)
        if (length_of(p.s, b) < 0)
          train::report_index(p.header, CHK_LENGTH, b, train::load_index(p.s.lens, b, p.s.id_bits), p.s.Sk);
  }
  const int l = threadIdx.x & 15;
  if (blockIdx.x >= row_blocks + pads) {
    const long long row = (long long)(blockIdx.x - row_blocks - pads) * 16 + (threadIdx.x >> 4);   // (batch, key, head)
    if (row >= (long long)p.s.B * p.s.Sk * p.s.Hk || 8 * l >= p.s.D) return;
    const int h = (int)(row % p.s.Hk), key = (int)(row / p.s.Hk % p.s.Sk), b = (int)(row / p.s.Hk / p.s.Sk);
    const int len = length_of(p.s, b);
    if (key < len && p.s.ntile > 0) return;
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = len < 0 ? NAN : 0.f;
    train::store_f32<__nv_bfloat16, 8>(p.dk + b * p.dk_b + key * p.dk_s + h * p.dk_h + 8 * l, t);
    train::store_f32<__nv_bfloat16, 8>(p.dv + b * p.dv_b + key * p.dv_s + h * p.dv_h + 8 * l, t);
    return;
  }
  if (blockIdx.x >= row_blocks) {
    const long long at = (long long)(blockIdx.x - row_blocks) * 256 + threadIdx.x;
    int token, head;
    if (at < (long long)p.s.B * p.s.Hk * p.s.ntile * kTile &&
        !row_of(p.s, (int)(at / kTile % p.s.ntile), (int)(at % kTile), token, head)) {
      p.delta[at] = 0.f;
      p.nnl[at] = -INFINITY;
    }
    return;
  }
  // (rows number less than 2^31)
  const unsigned rows = (unsigned)p.s.B * p.s.Sq * p.s.Hq;
  const unsigned row0 = (blockIdx.x * 16u + (threadIdx.x >> 4)) * kPreRows;
  train::Vec<__nv_bfloat16, 8> x[kPreRows], y[kPreRows];
#pragma unroll
  for (int k = 0; k < kPreRows; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k].w[i] = y[k].w[i] = 0u;
    if (row0 + k < rows && 8 * l < p.s.D) {
      x[k] = train::load_vec<__nv_bfloat16, 8>(p.o + (size_t)(row0 + k) * p.s.D + 8 * l);
      y[k] = train::load_vec<__nv_bfloat16, 8>(p.dO + (size_t)(row0 + k) * p.s.D + 8 * l);
    }
  }
  // the first row's place, then from head to head, token to token, batch to batch
  const unsigned bt = row0 / (unsigned)p.s.Hq;
  int b = (int)(bt / (unsigned)p.s.Sq), token = (int)(bt - (unsigned)b * p.s.Sq), h = (int)(row0 - bt * p.s.Hq);
  int hk = (unsigned)h / (unsigned)p.s.g, head = h - hk * p.s.g, tk = (unsigned)token / (unsigned)p.s.tpt;
  int i = token - tk * p.s.tpt;
#pragma unroll
  for (int k = 0; k < kPreRows; ++k) {
    float u[8], v[8], t = 0.f;
    train::unpack<__nv_bfloat16, 8>(x[k], u);
    train::unpack<__nv_bfloat16, 8>(y[k], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaf(u[e], v[e], t);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (row0 + k < rows) {
      if (l == 0) {
        const int tile = p.s.packed ? tk : head * p.s.nq + tk, r = p.s.packed ? i * p.s.g + head : i;
        const size_t at = ((size_t)(b * p.s.Hk + hk) * p.s.ntile + tile) * kTile + r;
        p.delta[at] = -t;
        const float nnl = -kLog2e * __ldg(p.lse + ((size_t)b * p.s.Hq + h) * p.s.Sq + token);
        p.nnl[at] = nnl == INFINITY ? -nnl : nnl;   // a row that sees nothing: P = 0
      }
      if ((p.s.lens || p.s.Sk == 0) && 8 * l < p.s.D) {
        const int len = length_of(p.s, b);
        if (len <= 0) {
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = len < 0 ? NAN : 0.f;
          train::store_f32<__nv_bfloat16, 8>(p.dq + b * p.dq_b + token * p.dq_s + h * p.dq_h + 8 * l, z);
        }
      }
    }
    ++h;
    if (++head == p.s.g) {
      head = 0;
      ++hk;
    }
    if (h == p.s.Hq) {
      h = hk = 0;
      ++token;
      if (++i == p.s.tpt) {
        i = 0;
        ++tk;
      }
      if (token == p.s.Sq) {
        token = tk = i = 0;
        ++b;
      }
    }
  }
}

template <int DT, bool DQ>
__global__ void __launch_bounds__(kThreads, 1)
    cross_keys_kernel(const __grid_constant__ BwdArgs p, const __grid_constant__ Maps maps) {
  using L = KeysLay<DT, DQ>;
  extern __shared__ __align__(1024) uint8_t smem_crossb[];
  uint8_t* sm = smem_crossb;
  uint64_t* bars = (uint64_t*)(sm + L::BAR_OFF);
  uint32_t* tmem_slot = (uint32_t*)(sm + L::BAR_OFF + 8 * C_COUNT);
  volatile int* abort_flag = (volatile int*)(sm + L::BAR_OFF + 8 * C_COUNT + 4);
  const int warp = same((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
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
      const bool both = (DQ && k == C_SP_FREE) || k == C_KV_EMPTY || k == C_ACC_FULL;   // issuers
      const bool rows = k >= C_DO_EMPTY && k < C_S_FULL;   // issuers and softmax-gradient warps
      const int n = k == C_P_FULL || k == C_DS_FULL ? 8 : k == C_DQ_EMPTY || k == C_ACC_EMPTY ? 4 : rows ? 10 : both ? 2 : 1;
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
  const uint32_t tmem = same(*tmem_slot);
  train::grid_wait();                              // Delta and LSE are there, the header is clear

  if (warp < 4) {
    ptx::regs_dec<L::REGS_SINGLE>();
    if (warp == 0 && lane == 0) {
      // ===================================== TMA producer =====================================
      KeysWalk<> w(p);
      int it = 0, tl = 0, loaded = 0;              // tasks, key tiles, dO tiles
      bool ok = !p.withhold;
      while (ok && w.next()) {
        const int qb = it % L::NQ;
        if (it >= L::NQ) ok = ptx::mbar_wait(bars + C_Q_EMPTY + qb, (it / L::NQ - 1) & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::mbar_expect_tx(bars + C_Q_FULL + qb, row_tile_bytes<DT>(p.s));
        load_row_tile<DT>(p.s, &maps.q, sm + L::Q_OFF + qb * L::TILE, w.at.b, w.at.hk, w.tile(), p.s.q_b, p.s.q_h,
                          bars + C_Q_FULL + qb);
        if (w.first_of_tile()) {
          if (tl > 0) ok = ptx::mbar_wait(bars + C_KV_EMPTY, (tl - 1) & 1, abort_flag, tmo);
          if (!ok) {
            ++it;
            break;
          }
          ptx::mbar_expect_tx(bars + C_KV_FULL, 2 * L::TILE);
          load_key_tile<DT>(&maps.k, sm + L::K_OFF, w.at.b, w.at.hk, w.at.d0, p.s.k_b, p.s.k_h, bars + C_KV_FULL);
          load_key_tile<DT>(&maps.v, sm + L::V_OFF, w.at.b, w.at.hk, w.at.d0, p.s.v_b, p.s.v_h, bars + C_KV_FULL);
          ++tl;
        }
        const int ob = it % L::NDO;
        if (it >= L::NDO) ok = ptx::mbar_wait(bars + C_DO_EMPTY + ob, (it / L::NDO - 1) & 1, abort_flag, tmo);
        if (!ok) {
          ++it;
          break;
        }
        const size_t row = ((size_t)w.group() * p.s.ntile + w.tile()) * kTile;
        uint8_t* offs = sm + L::OFFS_OFF + ob * L::OFFS;
        ptx::mbar_expect_tx(bars + C_DO_FULL + ob, row_tile_bytes<DT>(p.s) + L::OFFS);
        ptx::bulk_load(offs, p.nnl + row, kTile * 4, bars + C_DO_FULL + ob);
        ptx::bulk_load(offs + kTile * 4, p.delta + row, kTile * 4, bars + C_DO_FULL + ob);
        load_row_tile<DT>(p.s, &maps.dO, sm + L::DO_OFF + ob * L::TILE, w.at.b, w.at.hk, w.tile(), 1, 1,
                          bars + C_DO_FULL + ob);
        ++loaded;
        ++it;
      }
      // drain: every issued load has landed before the CTA may exit
      for (int k = max(0, it - L::NQ); k < it; ++k)
        ptx::mbar_drain(bars + C_Q_FULL + k % L::NQ, (k / L::NQ) & 1, 100000000ll);
      for (int k = max(0, loaded - L::NDO); k < loaded; ++k)
        ptx::mbar_drain(bars + C_DO_FULL + k % L::NDO, (k / L::NDO) & 1, 100000000ll);
      if (tl > 0) ptx::mbar_drain(bars + C_KV_FULL, (tl - 1) & 1, 100000000ll);
    } else if (warp == 2) {
      // ============================== key rows behind a length ================================
      KeysWalk<> w(p);
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
    } else if (warp == 1 || warp == 3) {
      // ==================================== MMA issuers =======================================
      // Warp 1 issues S^T and dV, warp 3 dP^T, dK and dQ^T, each in the tasks' order: so neither
      // chain waits in line behind the other's barriers.
      const uint32_t sK = ptx::smem_u32(sm + L::K_OFF), sV = ptx::smem_u32(sm + L::V_OFF);
      const uint32_t sQ = ptx::smem_u32(sm + L::Q_OFF), sdO = ptx::smem_u32(sm + L::DO_OFF);
      constexpr uint32_t ID_S = ptx::idesc_bf16(128, 128, 0, 0);
      const uint32_t id_ts = ptx::idesc_bf16(128, dsteps * 16, 0, 1);
      constexpr uint32_t BUF_STEP = L::TILE >> 4;
      // Every instruction between a product's end and the next one's start is time that the chain
      // loses (with all of a task's waits there: 700 cycles; 2630 us at 8192 x 8192 x 128, 32
      // heads, so 2550), so the walk and what else the next product waits for come before.
      KeysWalk<true> w(p);
      const uint32_t one = elect_one();
      int it = 0, tile = 0;                        // tasks and key tiles so far
      bool ok = true, more = w.next();
      if (warp == 1) {
        const uint32_t dK_k = ptx::sdesc_lo(sK, 16), dQ_k = ptx::sdesc_lo(sQ, 16);
        const uint32_t ddO_mn = ptx::sdesc_lo(sdO, kTile * 128);
        // S^T(it), once Q(it) has landed and what lies over its columns has been read: P^T(it-1) by dV,
        // with DQ also dS^T(it-1) by dK
        auto issue_s = [&](bool landed) {
          const int qb = it % L::NQ;
          if (!landed) {
            if (w.first_of_tile() && !ptx::warp_wait(bars + C_KV_READY, tile & 1, abort_flag, tmo)) return false;
            if (!ptx::warp_wait(bars + C_Q_FULL + qb, (it / L::NQ) & 1, abort_flag, tmo)) return false;
          }
          if (it > 0 && !ptx::warp_wait(bars + C_SP_FREE, (it - 1) & 1, abort_flag, tmo)) return false;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_SP, dK_k, dQ_k + qb * BUF_STEP, ID_S, dsteps, one);
          commit(bars + C_S_FULL, one);
          if (!DQ && one) ptx::mbar_arrive(bars + C_TURN + (it & 1));
          if (w.last_of_tile()) commit(bars + C_KV_EMPTY, one);
          return true;
        };
        if (more) ok = issue_s(false);
        while (ok && more) {
          const bool first = w.first_of_tile(), last = w.last_of_tile();
          const int ob = it % L::NDO;
          more = w.next();
          const bool landed = !last && is_complete(bars + C_Q_FULL + (it + 1) % L::NQ, ((it + 1) / L::NQ) & 1);
          // dV += P^T dO, once P^T(it) is stored and the last key tile's sums were read out
          ok = ptx::warp_wait(bars + C_DO_FULL + ob, (it / L::NDO) & 1, abort_flag, tmo);
          if (ok && first && tile > 0) ok = ptx::warp_wait(bars + C_ACC_EMPTY, (tile - 1) & 1, abort_flag, tmo);
          if (ok) ok = ptx::warp_wait(bars + C_P_FULL, it & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_rows<true>(tmem + L::T_DV, tmem + L::T_SP, ddO_mn + ob * BUF_STEP, id_ts, first ? 0u : 1u, 8, one);
          commit(bars + C_SP_FREE, one);
          commit(bars + C_DO_EMPTY + ob, one);
          if (last) {
            commit(bars + C_ACC_FULL, one);
            ++tile;
          }
          ++it;
          if (more) ok = issue_s(landed);
        }
      } else {
        const uint32_t dV_k = ptx::sdesc_lo(sV, 16), ddO_k = ptx::sdesc_lo(sdO, 16);
        const uint32_t dQ_mn = ptx::sdesc_lo(sQ, kTile * 128);
        const uint32_t dKt_mn = ptx::sdesc_lo(sK, DT == 128 ? kTile * 128 : L::ZERO_OFF - L::K_OFF);
        const uint32_t dDS_mn = ptx::sdesc_lo(ptx::smem_u32(sm + L::DS_OFF), kTile * 128);
        constexpr uint32_t ID_DQ = ptx::idesc_bf16(128, 128, 1, 1);
        // dP^T(it), once dO(it) has landed and its columns are free: dS^T(it-1) read by dK, with DQ
        // dQ^T(it-1) out of TMEM
        auto issue_dp = [&](bool landed) {
          const int ob = it % L::NDO;
          if (!landed) {
            if (w.first_of_tile() && !ptx::warp_wait(bars + C_KV_READY, tile & 1, abort_flag, tmo)) return false;
            if (!ptx::warp_wait(bars + C_DO_FULL + ob, (it / L::NDO) & 1, abort_flag, tmo)) return false;
          }
          if ((!DQ || !L::kSepDQ) && it > 0 &&
              !ptx::warp_wait(bars + (DQ ? C_DQ_EMPTY : C_DP_FREE), (it - 1) & 1, abort_flag, tmo))
            return false;
          ptx::tc_fence_after();
          issue_scores<DT>(tmem + L::T_DP, dV_k, ddO_k + ob * BUF_STEP, ID_S, dsteps, one);
          commit(bars + C_DP_FULL, one);
          commit(bars + C_DO_EMPTY + ob, one);
          if (w.last_of_tile() && !DQ) commit(bars + C_KV_EMPTY, one);
          return true;
        };
        if (more) ok = issue_dp(false);
        while (ok && more) {
          const bool first = w.first_of_tile(), last = w.last_of_tile();
          const int qb = it % L::NQ, ksteps = (w.keys() + 15) >> 4;
          more = w.next();
          const bool landed = !last && is_complete(bars + C_DO_FULL + (it + 1) % L::NDO, ((it + 1) / L::NDO) & 1);
          // dK += dS^T Q, once dS^T(it) is stored
          ok = ptx::warp_wait(bars + C_Q_FULL + qb, (it / L::NQ) & 1, abort_flag, tmo);
          if (ok && first && tile > 0) ok = ptx::warp_wait(bars + C_ACC_EMPTY, (tile - 1) & 1, abort_flag, tmo);
          if (ok) ok = ptx::warp_wait(bars + C_DS_FULL, it & 1, abort_flag, tmo);
          // The softmax waits for S^T(it+1) next, and that for dV(it): this chain's products get in line
          // behind both, for the time that the exponentials take. (Two barriers in turn: S^T(it+3)
          // cannot be issued before dP^T(it+1) is done.)
          if (!DQ && ok && !last) ok = ptx::warp_wait(bars + C_TURN + ((it + 1) & 1), ((it + 1) >> 1) & 1, abort_flag, tmo);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_rows<true>(tmem + L::T_DK, tmem + L::T_DS, dQ_mn + qb * BUF_STEP, id_ts, first ? 0u : 1u, 8, one);
          commit(bars + (DQ ? C_SP_FREE : C_DP_FREE), one);
          if (DQ) {
            // dQ^T = K^T dS^T
            if (L::kSepDQ && it > 0) ok = ptx::warp_wait(bars + C_DQ_EMPTY, (it - 1) & 1, abort_flag, tmo);
            if (!ok) break;
            ptx::tc_fence_after();
            issue_mn(tmem + L::T_DQ, dKt_mn, dDS_mn, ID_DQ, ksteps, one);
            commit(bars + C_DQ_FULL, one);
            if (last) commit(bars + C_KV_EMPTY, one);
          }
          commit(bars + C_Q_EMPTY + qb, one);
          if (last) {
            commit(bars + C_ACC_FULL, one);
            ++tile;
          }
          ++it;
          if (more) ok = issue_dp(landed);
        }
      }
      // drain: no MMA may be in flight when TMEM is released
      commit(bars + C_DRAIN + (warp >> 1), one);
      ptx::mbar_drain(bars + C_DRAIN + (warp >> 1), 0, 1000000000ll);
    }
  } else if (warp < 12) {
    // =============================== softmax-gradient warps =================================
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;             // key within the tile (TMEM lane)
    const int col0 = half * 64;                    // this thread's 64 rows
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    const uint32_t sDS = ptx::smem_u32(sm + L::DS_OFF);
    KeysWalk<> w(p);
    int it = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int ob = it % L::NDO;
      // (the offsets beside dO were copied by TMA: their own barrier is waited for as well)
      const float* nnl = (const float*)(sm + L::OFFS_OFF + ob * L::OFFS) + col0;
      const float* delta = nnl + kTile;
      ok = ptx::warp_wait(bars + C_DO_FULL + ob, (it / L::NDO) & 1, abort_flag, tmo);
      const bool pads = nnl[kTile - 1 - col0] == -INFINITY;   // rows that a tile does not have come last
      if (ok) ok = ptx::warp_wait(bars + C_S_FULL, it & 1, abort_flag, tmo);
      if (!ok) break;
      ptx::tc_fence_after();
      if (pads) {
        // (apart from the exponentials below, where any test takes 4 % of the kernel's time. Here the tiles that
        // have such rows pay: 4 x 300 rows x 2000 keys, 24 / 8 heads of 64, whose tiles all have: 87 us, now 92)
#pragma unroll 1
        for (int c0 = 0; c0 < 64; c0 += 16) {
          if (nnl[c0 + 15] != -INFINITY) continue;
          float s[16];
          ptx::tmem_ld16(tmem + lane_addr + L::T_SP + col0 + c0, s);
          uint32_t u[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(nnl[c0 + c] == -INFINITY ? 0.f : s[c]);
          ptx::tmem_st8(tmem + lane_addr + L::T_SP + col0 + c0, u);
          ptx::tmem_st8(tmem + lane_addr + L::T_SP + col0 + c0 + 8, u + 8);
        }
        ptx::tmem_wait_st();
      }
      float pv[64];
      {
        uint32_t a[32], b[32];
        ptx::tmem_ld32_issue(tmem + lane_addr + L::T_SP + col0, a);
        ptx::tmem_ld32_wait(a);
        ptx::tmem_ld32_issue(tmem + lane_addr + L::T_SP + col0 + 32, b);
        const uint64_t scale2 = two(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 f = *(const ulonglong2*)(nnl + c);
          exp2_two(__uint_as_float(a[c]), __uint_as_float(a[c + 1]), scale2, f.x, pv[c], pv[c + 1]);
          exp2_two(__uint_as_float(a[c + 2]), __uint_as_float(a[c + 3]), scale2, f.y, pv[c + 2], pv[c + 3]);
        }
        ptx::tmem_ld32_wait(b);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 f = *(const ulonglong2*)(nnl + 32 + c);
          exp2_two(__uint_as_float(b[c]), __uint_as_float(b[c + 1]), scale2, f.x, pv[32 + c], pv[33 + c]);
          exp2_two(__uint_as_float(b[c + 2]), __uint_as_float(b[c + 3]), scale2, f.y, pv[34 + c], pv[35 + c]);
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
      // dP^T(it) is complete; its commit covers dQ^T(it-1), the last reader of the shared dS^T tile
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
          const ulonglong2 f = *(const ulonglong2*)(delta + c0 + 2 * k);   // -Delta
          float x, y;
          untwo(mul2(two(pv[c0 + 2 * k], pv[c0 + 2 * k + 1]), add2(two(dp[2 * k], dp[2 * k + 1]), f.x)), x, y);
          u[k] = ptx::pack_bf16(x, y);
          untwo(mul2(two(pv[c0 + 2 * k + 2], pv[c0 + 2 * k + 3]), add2(two(dp[2 * k + 2], dp[2 * k + 3]), f.y)), x, y);
          u[k + 1] = ptx::pack_bf16(x, y);
        }
        ptx::tmem_st8(tmem + lane_addr + L::T_DS + col0 + c0 / 2, u);
        if (DQ) {
          store_chunk8(sDS, r, (col0 + c0) / 8, u);
          store_chunk8(sDS, r, (col0 + c0) / 8 + 1, u + 4);
        }
      }
      ptx::tmem_wait_st();
      if (DQ) ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bars + C_DS_FULL);
        ptx::mbar_arrive(bars + C_DO_EMPTY + ob);   // the offsets are read
      }
      ++it;
    }
  } else {
    // ======================= dQ read-out, and the epilogue of dK and dV ======================
    ptx::regs_inc<L::REGS_READOUT>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;           // d of dQ^T; key of dK and dV
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16);
    KeysWalk<> w(p);
    int it = 0, tl = 0;
    bool ok = true;
    while (ok && w.next()) {
      if constexpr (DQ) {
        ok = ptx::warp_wait(bars + C_DQ_FULL, it & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        float v[128];
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float t[32];
          ptx::tmem_ld32(tmem + lane_addr + L::T_DQ + c0, t);
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c0 + c] = t[c];
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + C_DQ_EMPTY);   // dQ^T(it) has left TMEM
        // Lanes 2k and 2k + 1 hold d = 2k and 2k + 1 of every row: the even lane takes both for even
        // rows, the odd lane for odd ones, so that a store has two of them.
        const int odd = lane & 1, d = row & ~1;
        int token, head;
        row_of(p.s, w.tile(), odd, token, head);
        __nv_bfloat16* dst = p.dq + w.at.b * p.dq_b + token * p.dq_s + (w.at.hk * p.s.g + head) * p.dq_h + d;
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
              head += 2;                           // two heads on, or into the next token
              dst += 2 * p.dq_h;
              if (head >= p.s.g) {
                head -= p.s.g;
                dst += p.dq_s - p.s.g * p.dq_h;
                --left;
              }
            }
          }
        }
      }
      if (w.last_of_tile()) {
        ok = ptx::warp_wait(bars + C_ACC_FULL, tl & 1, abort_flag, tmo);
        if (!ok) break;
        ptx::tc_fence_after();
        const int key = w.at.d0 * kTile + row;
        float* part = p.dkv_part + (((size_t)w.at.d1 * p.s.B * p.s.Hk + w.group()) * p.s.nk + w.at.d0) * 2 * kTile * DT;
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // dK, then dV
          const uint32_t from = tmem + lane_addr + (which ? L::T_DV : L::T_DK);
          __nv_bfloat16* dst = which ? p.dv + w.at.b * p.dv_b + key * p.dv_s + w.at.hk * p.dv_h
                                     : p.dk + w.at.b * p.dk_b + key * p.dk_s + w.at.hk * p.dk_h;
#pragma unroll
          for (int c0 = 0; c0 < DT; c0 += 32) {
            if (c0 < p.s.D) {
              float a[32];
              ptx::tmem_ld32(from + c0, a);
              if (p.qsegs > 1) store_part_32(part + which * kTile * DT, row, c0, a, 1.f);
              else store_rows_bf16(lane, a, which ? 1.f : p.scale, row < w.keys() ? dst + c0 : nullptr, p.s.D - c0);
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

// dk and dv of the keys within the lengths as the sums of the row segments' partials, in order; a thread
// takes 8 columns of a row.
template <int DT>
__global__ void __launch_bounds__(256) cross_join_keys_kernel(const __grid_constant__ BwdArgs p) {
  train::grid_next();
  train::grid_wait();
  const int per = p.s.D >> 3;
  const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
  const int c = (int)(item % per) * 8;
  const long long row = item / per;                // (batch, key, head)
  if (row >= (long long)p.s.B * p.s.Sk * p.s.Hk) return;
  const int h = (int)(row % p.s.Hk), key = (int)(row / p.s.Hk % p.s.Sk), b = (int)(row / p.s.Hk / p.s.Sk);
  if (key >= length_of(p.s, b)) return;
  const int kt = key / kTile;
  const float* src = p.dkv_part + ((((size_t)b * p.s.Hk + h) * p.s.nk + kt) * 2 * kTile) * DT + part_at(key % kTile, c);
  const size_t step = (size_t)p.s.B * p.s.Hk * p.s.nk * 2 * kTile * DT;
  float k[8] = {}, v[8] = {};
#pragma unroll 4
  for (int s = 0; s < p.qsegs; ++s) {
    float x[8], y[8];
    train::load_f32<float, 8>(src + s * step, x);
    train::load_f32<float, 8>(src + s * step + kTile * DT, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      k[i] += x[i];
      v[i] += y[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i] *= p.scale;
  train::store_f32<__nv_bfloat16, 8>(p.dk + b * p.dk_b + key * p.dk_s + h * p.dk_h + c, k);
  train::store_f32<__nv_bfloat16, 8>(p.dv + b * p.dv_b + key * p.dv_s + h * p.dv_h + c, v);
}

}  // namespace cross
}  // namespace dash
