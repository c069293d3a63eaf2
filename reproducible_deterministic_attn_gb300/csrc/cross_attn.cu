// Host side of cross attention (dash_cross_attn_*): argument checks, how the work is cut, tensor
// maps and launches. The kernels are in cross_fwd.cuh, cross_bwd.cuh and cross_bwd_rows.cuh.
#include <algorithm>
#include <atomic>
#include <climits>

#include "cross_bwd_rows.cuh"
#include "cross_fwd.cuh"
#include "dash_train.h"
#include "host_common.h"

namespace {

using namespace dash;
using namespace dash::cross;

// Work is cut for a chip of 152 SMs whatever the device has, so that equal arguments give equal
// bits everywhere.
constexpr int kChip = 152;

bool sizes_ok(int B, int Sq, int Sk, int Hq, int Hk, int D) {
  return B >= 1 && Sq >= 0 && Sk >= 0 && Hq >= 1 && Hk >= 1 && Hq % Hk == 0 && D >= 8 && D <= 128 && D % 8 == 0 &&
         B <= (1 << 20) && Hq <= (1 << 16) && Sq <= (1 << 24) && Sk <= (1 << 24) &&
         (long long)B * Hq * std::max(Sq, Sk) < (1ll << 31) - 256;
}

Shape make_shape(int B, int Sq, int Sk, int Hq, int Hk, int D, bool may_pack) {
  Shape s = {};
  s.B = B;
  s.Sq = Sq;
  s.Sk = Sk;
  s.Hq = Hq;
  s.Hk = Hk;
  s.g = Hq / Hk;
  s.D = D;
  s.nk = ceil_div(Sk, kTile);
  s.tpt = kTile;
  s.nq = ceil_div(Sq, kTile);
  s.ntile = s.nq * s.g;
  // all heads of a group in one row tile where that takes fewer tiles: 7 sequences' single tokens
  // with 4 heads a group are 56 tiles, not 224
  if (may_pack && s.g > 1 && s.g <= kTile) {
    const int tpt = kTile / s.g, n = ceil_div(Sq, tpt);
    if (n < s.ntile) {
      s.packed = 1;
      s.tpt = tpt;
      s.nq = s.ntile = n;
    }
  }
  return s;
}

// Key tiles that O or dQ sums in TMEM at most: the tensor core truncates its additions, so that sums of
// one sign come out small. Measured: O over 16384 keys by 1e-4, over these 65536 by 3.4e-4 (dQ by 4e-5), a
// twelfth of bf16's rounding; without a bound by 2 % over 4 M keys. Up to 65536 keys nothing is cut for it.
constexpr int kMaxKeyTiles = 512;

// Key ranges of the forward: as many as keep the units within one round of the chip, which takes at least two
// for each. Two where they make a second round cost more than they gain: 80 units of single tokens (5 x 16 key
// heads of 128) take 24 us with 1500 keys and 199 with 16384, in two ranges 29 and 204.
struct FwdPlan {
  int pairs, splits, kper;
  size_t part_o, part_l, total;      // workspace offsets and size
};
FwdPlan fwd_plan(const Shape& s) {
  FwdPlan p;
  p.pairs = ceil_div(s.ntile, 2);
  const long long units = (long long)s.B * s.Hk * p.pairs;
  p.splits = std::max(1, ceil_div(s.nk, kMaxKeyTiles));
  if (units > 0 && units * 2 <= kChip && s.nk > 1)
    p.splits = std::max(p.splits, (int)std::min<long long>(s.nk, kChip / units));
  p.kper = std::max(1, ceil_div(s.nk, p.splits));
  p.splits = std::max(1, ceil_div(s.nk, p.kper));
  const size_t rows = p.splits > 1 ? (size_t)p.splits * s.B * s.Hk * s.ntile * kTile : 0;
  p.part_o = kWsHeaderBytes;
  p.part_l = p.part_o + rows * (s.D <= 64 ? 64 : 128) * sizeof(float);
  p.total = round_up_to(p.part_l + rows * sizeof(float), 256);
  return p;
}

// {D, H, S, B} with element strides st = {batch, token, head}; dimensions of one place have one
// element and the coordinate 0.
bool map_heads(CUtensorMap* m, const void* ptr, int B, int S, int H, int D, const long long* st, int box_heads,
               int box_tokens) {
  const cuuint64_t pitch = (cuuint64_t)D * 2;
  const bool one_h = H == 1 || st[2] == 0, one_s = S == 1, one_b = B == 1 || st[0] == 0;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(one_h ? 1 : H), (cuuint64_t)S, (cuuint64_t)(one_b ? 1 : B)};
  const cuuint64_t strides[3] = {one_h ? pitch : (cuuint64_t)st[2] * 2, one_s ? pitch : (cuuint64_t)st[1] * 2,
                                 one_b ? pitch : (cuuint64_t)st[0] * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return dash::tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides,
                                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Element strides {batch, token, head} of a tensor that is read.
bool strides_ok(const long long* st, int S) {
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % 8 || st[i] > (1ll << 38)) return false;
  return S < 2 || st[1] > 0;
}

dash_status_t check(const void* q, const void* k, const void* v, const void* lens, const void* o, const float* lse,
                    int B, int Sq, int Sk, int Hq, int Hk, int D, const long long* qs, const long long* ks,
                    const long long* vs, float scale, int id_bits) {
  if (B < 0 || Sq < 0 || Sk < 0 || Hq < 1 || Hk < 1 || D < 1 || Hq % Hk) return DASH_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 3.4e38f)) return DASH_ERR_INVALID_ARG;
  if (id_bits != 32 && id_bits != 64) return DASH_ERR_INVALID_ARG;
  if (B > 0 && !sizes_ok(B, Sq, Sk, Hq, Hk, D)) return DASH_ERR_UNSUPPORTED;
  if (!qs || !ks || !vs) return DASH_ERR_INVALID_ARG;
  if (!strides_ok(qs, Sq) || !strides_ok(ks, Sk) || !strides_ok(vs, Sk)) return DASH_ERR_UNSUPPORTED;
  const bool rows = (long long)B * Sq > 0, keys = (long long)B * Sk > 0;
  if ((rows && (!q || !o || !lse)) || (keys && (!k || !v))) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(o, 16) || !is_aligned(lse, 4) ||
      !is_aligned(lens, id_bits / 8))
    return DASH_ERR_INVALID_ARG;
  return DASH_OK;
}

dash_status_t bad_map() {
  dash::set_last_error(dash::tensor_map_encoder() ? "cuTensorMapEncodeTiled rejected a tensor"
                                                  : "cuTensorMapEncodeTiled is not available from the driver");
  return DASH_ERR_CUDA;
}

dash_status_t sm_count(int* sms) {
  int dev = 0;
  DASH_TRY(cudaGetDevice(&dev));
  DASH_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return DASH_OK;
}

// Shared memory of a kernel that moves registers between its warpgroups: their shares add up to
// what it was launched with only if it was built with exactly that count.
// (`known`: a bit for each device that has been asked.)
dash_status_t prepare(const void* kernel, int smem, int regs, std::atomic<uint64_t>* known) {
  int dev = 0;
  DASH_TRY(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (known->load(std::memory_order_acquire) & bit) return DASH_OK;
  cudaFuncAttributes fa;
  DASH_TRY(cudaFuncGetAttributes(&fa, kernel));
  if (fa.numRegs != regs) {
    dash::set_last_error("cross attention kernel was not built with the register count its warp roles share");
    return DASH_ERR_CUDA;
  }
  DASH_TRY(dash::allow_shared(kernel, smem));
  known->fetch_or(bit, std::memory_order_release);
  return DASH_OK;
}

// A tensor without elements still needs a map: any readable place will do, as no tile is loaded.
bool make_maps(Maps* m, const Shape& s, const void* q, const void* k, const void* v, const long long* qs,
               const long long* ks, const long long* vs) {
  const int bh = s.packed ? s.g : 1, bt = s.packed ? s.tpt : kTile;
  if (!dash::tensor_map_encoder()) return false;
  if (!map_heads(&m->q, q, s.B, s.Sq, s.Hq, s.D, qs, bh, bt)) return false;
  if (s.Sk == 0) return true;
  return map_heads(&m->k, k, s.B, s.Sk, s.Hk, s.D, ks, 1, kTile) &&
         map_heads(&m->v, v, s.B, s.Sk, s.Hk, s.D, vs, 1, kTile);
}

void set_places(Shape* s, const long long* qs, const long long* ks, const long long* vs) {
  s->q_b = qs[0] != 0;
  s->q_h = qs[2] != 0;
  s->k_b = ks[0] != 0;
  s->k_h = ks[2] != 0;
  s->v_b = vs[0] != 0;
  s->v_h = vs[2] != 0;
}

// The units of a kernel whose fastest digits are d0 and d1, and the CTAs that share them.
Units make_units(const Shape& s, int d0, int d1, int sms, int* grid) {
  Units n = {};
  n.radix[0] = d0;
  n.radix[1] = s.Hk;
  n.radix[2] = d1;
  n.batches = s.B;
  const long long all = (long long)d0 * d1 * s.Hk * s.B;
  *grid = (int)std::min<long long>(all, sms);
  int g = *grid;
  for (int i = 0; i < 3; ++i) {
    n.step[i] = g % n.radix[i];
    g /= n.radix[i];
  }
  n.step[3] = g;
  return n;
}

template <int DT>
dash_status_t launch_fwd(FwdArgs a, const Maps& maps, cudaStream_t stream) {
  static std::atomic<uint64_t> known{0};
  const dash_status_t st = prepare((const void*)cross_fwd_kernel<DT>, FwdLay<DT>::ALLOC, kFwdRegsLaunch, &known);
  if (st != DASH_OK) return st;
  int sms = 0;
  if (const dash_status_t e = sm_count(&sms)) return e;
  int grid = 0;
  a.units = make_units(a.s, a.splits, a.pairs, sms, &grid);
  cross_fwd_kernel<DT><<<grid, kFwdThreads, FwdLay<DT>::ALLOC, stream>>>(a, maps);
  DASH_TRY(cudaGetLastError());
  if (a.splits > 1) {
    const long long rows = (long long)a.s.B * a.s.Hk * a.s.ntile * kTile;
    DASH_TRY(dash::launch_after(cross_join_kernel<DT>, dim3((unsigned)ceil_div<long long>(rows, 8)), 256, 0, stream, a));
  }
  return DASH_OK;
}

// Strides of a tensor to write: no two of its elements in one place by a stride of zero.
bool distinct(const long long* st, int B, int S, int H) {
  return (B < 2 || st[0] > 0) && (S < 2 || st[1] > 0) && (H < 2 || st[2] > 0);
}

// How the backward is cut: cross_keys_kernel's row segments and cross_rows_kernel's key segments.
// Every cut costs partials (written and read once more) and the start of another unit, too few leave
// SMs idle, so each is the cheapest by a count of tasks of 128 x 128 scores: a unit takes its tasks
// and `start` more, units run in rounds of the chip, and partials cost what memory takes for them (a
// task is about 1.5 us, in which the chip moves 10 MB). Where batches have lengths of their own, which
// the host does not know, a fifth of the units is taken to be empty. A row segment has at most 128
// row tiles, as the tensor core's truncation loses at most 2^-15.5 of a sum of one sign over them (a key
// range at most kMaxKeyTiles).
int best_cut(long long units, int tasks, int least, double start, double part_bytes, bool ragged) {
  int cut = least;
  double best = 1e300;
  for (int n = least; n <= tasks; ++n) {
    const int per = ceil_div(tasks, n);
    if (ceil_div(tasks, per) != n) continue;
    const double rounds = (double)ceil_div<long long>(ragged ? ceil_div<long long>(4 * units * n, 5) : units * n, kChip);
    const double cost = rounds * (per + start) + (n > 1 ? 1 + 2 * n * part_bytes / 10e6 : 0.0);
    if (cost < best) {
      best = cost;
      cut = n;
    }
    if (units * n > 8 * kChip) break;
  }
  return cut;
}
struct BwdPlan {
  bool one;                          // one key tile: cross_keys_kernel forms dQ too
  int qsegs, qper, ksegs, kper;
  size_t nnl, delta, dq_part, dkv_part, total;
};
BwdPlan bwd_plan(const Shape& s, bool ragged) {
  BwdPlan p = {};
  const long long groups = (long long)s.B * s.Hk;
  const int nt = s.ntile, nk = s.nk, dt = s.D <= 64 ? 64 : 128;
  const size_t rows = (size_t)groups * nt * kTile, keys = (size_t)groups * nk * kTile;
  p.one = nk == 1;
  p.qsegs = p.ksegs = p.qper = p.kper = 1;
  if (nt > 0 && nk > 0) {
    p.qsegs = best_cut(groups * nk, nt, ceil_div(nt, 128), 2, (double)keys * dt * 8, ragged);
    p.qper = ceil_div(nt, p.qsegs);
    if (!p.one) {
      p.ksegs = best_cut(groups * nt, nk, ceil_div(nk, kMaxKeyTiles), 2, (double)rows * dt * 4, ragged);
      p.kper = ceil_div(nk, p.ksegs);
    }
  }
  p.nnl = kWsHeaderBytes;
  p.delta = p.nnl + rows * sizeof(float);
  p.dq_part = round_up_to(p.delta + rows * sizeof(float), 256);
  p.dkv_part = p.dq_part + (p.ksegs > 1 ? p.ksegs * rows * dt * sizeof(float) : 0);
  p.total = p.dkv_part + (p.qsegs > 1 ? p.qsegs * keys * 2 * dt * sizeof(float) : 0);
  p.total = round_up_to(std::max(p.total, kWsHeaderBytes), 256);
  return p;
}

template <int DT, bool DQ>
dash_status_t launch_keys(BwdArgs a, const Maps& maps, int sms, cudaStream_t stream) {
  using L = KeysLay<DT, DQ>;
  static std::atomic<uint64_t> known{0};
  const dash_status_t st = prepare((const void*)cross_keys_kernel<DT, DQ>, L::ALLOC, L::REGS_LAUNCH, &known);
  if (st != DASH_OK) return st;
  int grid = 0;
  a.units = make_units(a.s, a.s.nk, a.qsegs, sms, &grid);
  DASH_TRY(dash::launch_after(cross_keys_kernel<DT, DQ>, dim3(grid), kThreads, L::ALLOC, stream, a, maps));
  return DASH_OK;
}

template <int DT>
dash_status_t launch_bwd(BwdArgs a, bool one, const Maps& maps, cudaStream_t stream) {
  int sms = 0;
  if (const dash_status_t e = sm_count(&sms)) return e;
  const long long rows = (long long)a.s.B * a.s.Hk * a.s.ntile * kTile;
  const bool work = a.s.ntile > 0 && a.s.nk > 0;
  const unsigned row_blocks =
      (unsigned)std::max(1ll, ceil_div<long long>((long long)a.s.B * a.s.Sq * a.s.Hq, 16 * kPreRows));
  // places of row tiles without a row: behind the last token, and where heads fill no tile
  const bool padded = a.s.Sq % a.s.tpt || (a.s.packed && a.s.g * a.s.tpt < kTile);
  const unsigned pads = padded ? (unsigned)ceil_div<long long>(rows, 256) : 0;
  // keys that no unit's sums go to: behind lengths, or all where there are no rows
  const unsigned key_blocks =
      a.s.lens || !work ? (unsigned)ceil_div<long long>((long long)a.s.B * a.s.Sk * a.s.Hk, 16) : 0;
  cross_pre_kernel<<<row_blocks + pads + key_blocks, 256, 0, stream>>>(a, row_blocks, pads);
  DASH_TRY(cudaGetLastError());
  if (!work) return DASH_OK;
  if (const dash_status_t e = one ? launch_keys<DT, true>(a, maps, sms, stream)
                                  : launch_keys<DT, false>(a, maps, sms, stream))
    return e;
  const int per = a.s.D / 8;
  if (a.qsegs > 1) {
    const unsigned blocks = (unsigned)ceil_div<long long>((long long)a.s.B * a.s.Sk * a.s.Hk * per, 256);
    DASH_TRY(dash::launch_after(cross_join_keys_kernel<DT>, dim3(blocks), 256, 0, stream, a));
  }
  if (!one) {
    static std::atomic<uint64_t> known{0};
    const dash_status_t st = prepare((const void*)cross_rows_kernel<DT>, RowsLay<DT>::ALLOC, kRowsRegsLaunch, &known);
    if (st != DASH_OK) return st;
    int grid = 0;
    a.units = make_units(a.s, a.ksegs, a.s.ntile, sms, &grid);
    DASH_TRY(dash::launch_after(cross_rows_kernel<DT>, dim3(grid), kRowsThreads, RowsLay<DT>::ALLOC,
                                stream, a, maps));
    if (a.ksegs > 1)
      DASH_TRY(dash::launch_after(cross_join_rows_kernel<DT>, dim3((unsigned)ceil_div<long long>(rows * per, 256)), 256,
                                  0, stream, a));
  }
  return DASH_OK;
}

}  // namespace

extern "C" {

size_t dash_cross_attn_fwd_workspace_size(int B, int Sq, int Sk, int Hq, int Hk, int D) {
  if (!sizes_ok(B, Sq, Sk, Hq, Hk, D)) return 0;
  return std::max(fwd_plan(make_shape(B, Sq, Sk, Hq, Hk, D, true)).total,
                  fwd_plan(make_shape(B, Sq, Sk, Hq, Hk, D, false)).total);
}

dash_status_t dash_cross_attn_fwd(const void* q, const void* k, const void* v, const void* kv_lens, void* o,
                                  float* lse, int* status, void* workspace, size_t workspace_bytes, int B, int Sq,
                                  int Sk, int Hq, int Hk, int D, const long long* q_strides,
                                  const long long* k_strides, const long long* v_strides, float scale, int id_bits,
                                  cudaStream_t stream) {
  const dash_status_t st = check(q, k, v, kv_lens, o, lse, B, Sq, Sk, Hq, Hk, D, q_strides, k_strides, v_strides,
                                 scale, id_bits);
  if (st != DASH_OK) return st;
  if (!is_aligned(status, 4) || !is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  FwdArgs a = {};
  a.s = make_shape(B, Sq, Sk, Hq, Hk, D, q_strides[2] != 0);
  a.s.lens = kv_lens;
  a.s.id_bits = id_bits;
  set_places(&a.s, q_strides, k_strides, v_strides);
  const FwdPlan pl = fwd_plan(a.s);
  if (pl.splits > 1) {
    if (!workspace) return DASH_ERR_INVALID_ARG;
    if (workspace_bytes < pl.total) return DASH_ERR_WORKSPACE_TOO_SMALL;
    a.part_o = (float*)((char*)workspace + pl.part_o);
    a.part_l = (float*)((char*)workspace + pl.part_l);
  }
  a.o = (__nv_bfloat16*)o;
  a.lse = lse;
  a.pairs = pl.pairs;
  a.splits = pl.splits;
  a.kper = pl.kper;
  a.scale_log2 = scale * kLog2e;
  a.status = status;
  a.timeout_ns = sync_timeout_ns();
  a.withhold = sync_withheld();
  if (status) DASH_TRY(cudaMemsetAsync(status, 0, sizeof(int), stream));
  if ((long long)B * Sq == 0) return DASH_OK;
  Maps maps;
  if (!make_maps(&maps, a.s, q, k, v, q_strides, k_strides, v_strides)) return bad_map();
  return D <= 64 ? launch_fwd<64>(a, maps, stream) : launch_fwd<128>(a, maps, stream);
}

size_t dash_cross_attn_bwd_workspace_size(int B, int Sq, int Sk, int Hq, int Hk, int D) {
  if (!sizes_ok(B, Sq, Sk, Hq, Hk, D)) return 0;
  size_t most = 0;
  for (bool pack : {false, true})
    for (bool ragged : {false, true})
      most = std::max(most, bwd_plan(make_shape(B, Sq, Sk, Hq, Hk, D, pack), ragged).total);
  return most;
}

dash_status_t dash_cross_attn_bwd(const void* q, const void* k, const void* v, const void* kv_lens, const void* o,
                                  const void* d_o, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                                  size_t workspace_bytes, int B, int Sq, int Sk, int Hq, int Hk, int D,
                                  const long long* q_strides, const long long* k_strides,
                                  const long long* v_strides, const long long* dq_strides,
                                  const long long* dk_strides, const long long* dv_strides, float scale,
                                  int id_bits, cudaStream_t stream) {
  const dash_status_t st = check(q, k, v, kv_lens, o, lse, B, Sq, Sk, Hq, Hk, D, q_strides, k_strides, v_strides,
                                 scale, id_bits);
  if (st != DASH_OK) return st;
  if (!dq_strides || !dk_strides || !dv_strides || !workspace) return DASH_ERR_INVALID_ARG;
  if (!strides_ok(dq_strides, Sq) || !strides_ok(dk_strides, Sk) || !strides_ok(dv_strides, Sk))
    return DASH_ERR_UNSUPPORTED;
  if (!distinct(dq_strides, B, Sq, Hq) || !distinct(dk_strides, B, Sk, Hk) || !distinct(dv_strides, B, Sk, Hk))
    return DASH_ERR_INVALID_ARG;
  if (((long long)B * Sq > 0 && (!d_o || !dq)) || ((long long)B * Sk > 0 && (!dk || !dv))) return DASH_ERR_INVALID_ARG;
  for (const void* t : {d_o, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!is_aligned(t, 16)) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  if (workspace_bytes < kWsHeaderBytes) return DASH_ERR_WORKSPACE_TOO_SMALL;
  if (B == 0) {
    DASH_TRY(cudaMemsetAsync(workspace, 0, kWsHeaderBytes, stream));
    return DASH_OK;
  }
  BwdArgs a = {};
  a.s = make_shape(B, Sq, Sk, Hq, Hk, D, q_strides[2] != 0);
  a.s.lens = kv_lens;
  a.s.id_bits = id_bits;
  set_places(&a.s, q_strides, k_strides, v_strides);
  const BwdPlan pl = bwd_plan(a.s, kv_lens != nullptr);
  if (workspace_bytes < pl.total) return DASH_ERR_WORKSPACE_TOO_SMALL;
  char* ws = (char*)workspace;
  a.header = (int*)ws;
  a.nnl = (float*)(ws + pl.nnl);
  a.delta = (float*)(ws + pl.delta);
  a.dq_part = (float*)(ws + pl.dq_part);
  a.dkv_part = (float*)(ws + pl.dkv_part);
  a.o = (const __nv_bfloat16*)o;
  a.dO = (const __nv_bfloat16*)d_o;
  a.lse = lse;
  a.dq = (__nv_bfloat16*)dq;
  a.dk = (__nv_bfloat16*)dk;
  a.dv = (__nv_bfloat16*)dv;
  a.dq_b = dq_strides[0];
  a.dq_s = dq_strides[1];
  a.dq_h = dq_strides[2];
  a.dk_b = dk_strides[0];
  a.dk_s = dk_strides[1];
  a.dk_h = dk_strides[2];
  a.dv_b = dv_strides[0];
  a.dv_s = dv_strides[1];
  a.dv_h = dv_strides[2];
  a.qsegs = pl.qsegs;
  a.qper = pl.qper;
  a.ksegs = pl.ksegs;
  a.kper = pl.kper;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.timeout_ns = sync_timeout_ns();
  a.withhold = sync_withheld();
  Maps maps;
  if (Sq > 0 && Sk > 0) {
    const long long os[3] = {(long long)Sq * Hq * D, (long long)Hq * D, (long long)D};
    const int bh = a.s.packed ? a.s.g : 1, bt = a.s.packed ? a.s.tpt : kTile;
    if (!make_maps(&maps, a.s, q, k, v, q_strides, k_strides, v_strides) ||
        !map_heads(&maps.dO, d_o, B, Sq, Hq, D, os, bh, bt))
      return bad_map();
  }
  return D <= 64 ? launch_bwd<64>(a, pl.one, maps, stream) : launch_bwd<128>(a, pl.one, maps, stream);
}

}  // extern "C"
