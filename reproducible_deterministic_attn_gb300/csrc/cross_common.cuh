// Cross attention (dash_cross_attn_*): what the forward and the backward share.
//
// Queries [B, Sq, Hq, D] look at keys [B, Sk, Hk, D] of another length, of which batch b has the
// first len_b. The g = Hq / Hk query heads that share a key head form a group; the query rows of
// a group are cut into row tiles of up to 128 rows, one TMEM lane each. A row tile is 128
// consecutive tokens of one head, or (packed, chosen where it takes fewer tiles, as for single
// tokens) 128 / g consecutive tokens with all g heads: row = token * g + head, which a 4-D tensor
// map loads as one box. Tensors are read through 4-D maps {D, head, token, batch}, so rows and
// columns beyond a tensor's extent arrive as zeros and strides need only be multiples of 16 bytes.
#pragma once

#include "bwd_main.cuh"
#include "tc_shared.cuh"
#include "train_common.cuh"

namespace dash {
namespace cross {

using namespace dash::tc;

struct Shape {
  int B, Sq, Sk, Hq, Hk, g, D;
  int packed;                // row tiles hold all heads of a group
  int tpt;                   // tokens of a row tile (128, or 128 / g when packed)
  int nq;                    // row tiles along the tokens
  int ntile;                 // row tiles of a group: nq, times g when not packed
  int nk;                    // key tiles of 128
  // 1, or 0 where a tensor's batches or heads lie in one place (a stride of zero)
  int q_b, q_h, k_b, k_h, v_b, v_h;
  const void* lens;          // [B], or null: every length is Sk
  int id_bits;
};

struct Maps {
  CUtensorMap q, k, v, dO;   // 4-D bf16 {D, H, S, B}
};

// Units of work number a kernel's [batch][d1][key head][d0]; a CTA takes every grid-th. The heads lie
// side by side, so that CTAs that run together read a token's heads, whole lines of memory, together
// (8192 x 512, 16 heads of 128, forward: 75 us with the heads behind d1, then 71). Nothing is asked of
// L2 ahead of time: such requests took the copies' own turns (68 us without them). A CTA steps from
// unit to unit digit by digit, as a division takes more than all of a step.
struct Units {
  int radix[3];              // of d0, the key heads, d1
  int step[4];               // the grid's digits
  int batches;
};
struct Place {
  int d0, d1, hk, b;
  __device__ __forceinline__ Place(const Units& n) {
    int u = (int)blockIdx.x;
    d0 = u % n.radix[0];
    u /= n.radix[0];
    hk = u % n.radix[1];
    u /= n.radix[1];
    d1 = u % n.radix[2];
    b = u / n.radix[2];
  }
  __device__ __forceinline__ bool more(const Units& n) const { return b < n.batches; }
  __device__ __forceinline__ void next(const Units& n) {
    d0 += n.step[0];
    const int c0 = d0 >= n.radix[0];
    d0 -= c0 ? n.radix[0] : 0;
    hk += n.step[1] + c0;
    const int c1 = hk >= n.radix[1];
    hk -= c1 ? n.radix[1] : 0;
    d1 += n.step[2] + c1;
    const int c2 = d1 >= n.radix[2];
    d1 -= c2 ? n.radix[2] : 0;
    b += n.step[3] + c2;
  }
};

// The batch's number of keys; -1 when it is out of range (treated as none).
__device__ __forceinline__ int length_of(const Shape& s, int b) {
  if (!s.lens) return s.Sk;
  const long long n = train::load_index(s.lens, b, s.id_bits);
  return n >= 0 && n <= s.Sk ? (int)n : -1;
}

// Row r of row tile t of a group: its token and its head within the group; false where the tile
// has no such row.
__device__ __forceinline__ bool row_of(const Shape& s, int t, int r, int& token, int& head) {
  if (s.packed) {
    const int i = r / s.g;
    token = t * s.tpt + i;
    head = r - i * s.g;
    return i < s.tpt && token < s.Sq;
  }
  head = t / s.nq;
  token = (t - head * s.nq) * kTile + r;
  return token < s.Sq;
}

// Loads the 64-column blocks of row tile t into shared memory, `rows` of 128 bytes each.
template <int DT>
__device__ __forceinline__ uint32_t row_tile_bytes(const Shape& s) {
  return (uint32_t)(DT / 64) * 128u * (s.packed ? (uint32_t)(s.g * s.tpt) : (uint32_t)kTile);
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(ptx::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(ptx::smem_u32(bar))
      : "memory");
}
template <int DT>
__device__ __forceinline__ void load_row_tile(const Shape& s, const CUtensorMap* map, uint8_t* dst, int b, int hk,
                                              int t, int mul_b, int mul_h, uint64_t* bar) {
  int head = 0, token = t * s.tpt;
  if (!s.packed) {
    head = t / s.nq;
    token = (t - head * s.nq) * kTile;
  }
#pragma unroll
  for (int cb = 0; cb < DT / 64; ++cb)
    tma_load_4d(dst + cb * kTile * 128, map, cb * 64, (hk * s.g + head) * mul_h, token, b * mul_b, bar);
}
template <int DT>
__device__ __forceinline__ void load_key_tile(const CUtensorMap* map, uint8_t* dst, int b, int hk, int t, int mul_b,
                                              int mul_h, uint64_t* bar) {
#pragma unroll
  for (int cb = 0; cb < DT / 64; ++cb)
    tma_load_4d(dst + cb * kTile * 128, map, cb * 64, hk * mul_h, t * kTile, b * mul_b, bar);
}

// Whether a phase is complete, without waiting; the warp agrees.
__device__ __forceinline__ bool is_complete(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(ptx::smem_u32(bar)), "r"(parity)
               : "memory");
  return __all_sync(0xffffffffu, done) != 0;
}

// Products are issued by a warp that stays together, of whose lanes one (`one` != 0) issues: so
// descriptors and barriers' addresses stay in uniform registers. Issued by a lone thread each step
// moves its operands there one by one, among the softmax warps that share its scheduler: two
// products of 128 x 128 x 128 took 1900 to 3100 cycles beside busy warps instead of 1024 to 1530.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one;
}
__device__ __forceinline__ uint32_t same(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t one) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 da, db; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %6, 0; mov.b64 da, {%1, %5}; "
      "mov.b64 db, {%2, %5}; @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(ptx::kDescHi), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t one) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 db; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %6, 0; mov.b64 db, {%2, %5}; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(ptx::kDescHi), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0; "
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(ptx::smem_u32(bar)),
      "r"(one)
      : "memory");
}

// The K steps of 16 of a product, n of them. Two K-major operands in shared memory (64 columns a
// block of 128 rows):
template <int DT>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int n, uint32_t one) {
#pragma unroll
  for (int ks = 0; ks < DT / 16; ++ks) {
    const uint32_t step = ((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4;
    if (ks < n) mma_ss(d, a + step, b + step, id, ks > 0, one);
  }
}
// A in TMEM, 16 of K in 8 packed columns, side by side or (SPLIT) in two halves whose bases are 64
// apart; B MN-major in shared memory:
template <bool SPLIT>
__device__ __forceinline__ void issue_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc0, int n,
                                           uint32_t one) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    if (ks < n) mma_ts(d, a + (SPLIT ? 64 * (ks >> 2) + 8 * (ks & 3) : 8 * ks), b + ks * kMnStep, id, ks > 0 ? 1u : acc0, one);
}
// Both operands MN-major in shared memory:
__device__ __forceinline__ void issue_mn(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int n, uint32_t one) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    if (ks < n) mma_ss(d, a + ks * kMnStep, b + ks * kMnStep, id, ks > 0, one);
}

// Zeroes rows [from, to) of a tile in shared memory (one warp): keys that a length leaves out may
// hold anything, and 0 * NaN in a product over the keys would be NaN.
template <int DT>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int lane) {
  const int pieces = (to - from) * 8;              // of 16 bytes, in each 64-column block
#pragma unroll
  for (int cb = 0; cb < DT / 64; ++cb)
    for (int i = lane; i < pieces; i += 32)
      reinterpret_cast<uint4*>(tile + cb * kTile * 128 + from * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
}

using train::add2;
using train::fma2;
using train::mul2;
using train::two;
using train::untwo;
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// exp2(x scale + offset) of two values
__device__ __forceinline__ void exp2_two(float x, float y, uint64_t scale, uint64_t offset, float& ex, float& ey) {
  float u, v;
  untwo(fma2(two(x, y), scale, offset), u, v);
  ex = ptx::ex2(u);
  ey = ptx::ex2(v);
}

// 32 columns of a warp's 32 rows, a row a thread (times f, n of the columns valid, a multiple of 8;
// dst null: no such row), to global memory as bf16. Four lanes swap 16-byte pieces of their rows, so
// that they store 64 bytes of a row side by side: 32 bytes of 32 rows in one store took a cycle for
// each row's line, 5000 cycles for a pair of tiles of 128 columns.
__device__ __forceinline__ void swap_pieces(uint4& a, uint4& b, bool high, int lanes) {
  uint4 x = high ? a : b;
  x.x = __shfl_xor_sync(0xffffffffu, x.x, lanes);
  x.y = __shfl_xor_sync(0xffffffffu, x.y, lanes);
  x.z = __shfl_xor_sync(0xffffffffu, x.z, lanes);
  x.w = __shfl_xor_sync(0xffffffffu, x.w, lanes);
  if (high) a = x;
  else b = x;
}
__device__ __forceinline__ void store_rows_bf16(int lane, const float (&v)[32], float f, __nv_bfloat16* dst, int n) {
  uint4 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = make_uint4(ptx::pack_bf16(v[8 * i] * f, v[8 * i + 1] * f), ptx::pack_bf16(v[8 * i + 2] * f, v[8 * i + 3] * f),
                      ptx::pack_bf16(v[8 * i + 4] * f, v[8 * i + 5] * f), ptx::pack_bf16(v[8 * i + 6] * f, v[8 * i + 7] * f));
  swap_pieces(c[0], c[1], lane & 1, 1);
  swap_pieces(c[2], c[3], lane & 1, 1);
  swap_pieces(c[0], c[2], lane & 2, 2);
  swap_pieces(c[1], c[3], lane & 2, 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {                    // piece `lane & 3` of row i of the four
    __nv_bfloat16* to = (__nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)dst, (lane & ~3) + i);
    if (to && 8 * (lane & 3) < n) *reinterpret_cast<uint4*>(to + 8 * (lane & 3)) = c[i];
  }
}

// fp32 partials of a tile lie 8 columns of every row side by side, [DT / 8][128][8], so that a warp's
// stores are whole lines and a row's reads whole sectors: column c (a multiple of 8) of row r is at
__device__ __forceinline__ size_t part_at(int r, int c) { return (size_t)(c * kTile + r * 8); }
// 32 columns from c0 (times f) of row r.
__device__ __forceinline__ void store_part_32(float* tile, int r, int c0, const float (&v)[32], float f) {
#pragma unroll
  for (int c = 0; c < 32; c += 8)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(tile + part_at(r, c0 + c)),
                 "f"(v[c] * f), "f"(v[c + 1] * f), "f"(v[c + 2] * f), "f"(v[c + 3] * f), "f"(v[c + 4] * f),
                 "f"(v[c + 5] * f), "f"(v[c + 6] * f), "f"(v[c + 7] * f)
                 : "memory");
}

}  // namespace cross
}  // namespace dash
