// C ABI of the cross entropy from hidden states (dash_linear_xent_*): argument checks, the
// pieces of the vocabulary, workspace layout and launches.
#include <algorithm>

#include "dash_train.h"
#include "host_common.h"
#include "linear_xent.cuh"

namespace {

using namespace dash::xent;
using dash::ceil_div;
using dash::is_aligned;
using dash::round_up_to;

// Vocabulary rows of one piece of the backward: G [T, piece] bf16 takes at most this many
// bytes (a piece is at least one 256-column tile).
constexpr size_t kPieceBytes = 256ull << 20;
constexpr int kMinSplitKSteps = 8;      // a K range of dX is at least 512 wide
constexpr int kSplitTarget = 76;        // units that a split dX aims for (one GB300's pairs of SMs)

struct Plan {
  long long piece;            // vocabulary rows a piece, a multiple of 256
  int pieces;
  long long ldg;
  bool two;                   // up to kTwoTermRows tokens: G's two terms share DX's tiles
  long long g2_rows;          // rows from G's first terms to its second ones (0: there are none)
  long long dx_rows;          // rows of one K range's dX
  int dx_splits, dx_ksteps;   // K ranges of dX within a full piece
  bool joined;                // dX goes through partials and a join
  size_t part, ztgt;          // forward
  size_t g, acc, dx_part;     // backward
  size_t total;
};

bool sizes_ok(long long T, long long V, int D) {
  const long long lim = (1ll << 31) - 256;
  return T >= 0 && V >= 1 && D >= 8 && D % 8 == 0 && T < lim && V < lim &&
         T * D <= (1ll << 40) && V * D <= (1ll << 40);
}

// dX's K ranges: one when its tiles fill the grid, else as many as give kSplitTarget units,
// each at least kMinSplitKSteps steps of 64. Depends on the sizes alone.
void dx_ranges(long long T, int D, long long piece, int* splits, int* per) {
  const long long tiles = ceil_div<long long>(T, kTM) * ceil_div<long long>(D, kTN);
  const int steps = (int)ceil_div<long long>(piece, kTK);
  long long s = tiles > 0 ? kSplitTarget / tiles : 1;
  s = std::max<long long>(1, std::min<long long>(s, steps / kMinSplitKSteps));
  *per = (int)ceil_div<long long>(steps, s);
  *splits = (int)ceil_div<long long>(steps, *per);
}

Plan make_plan(long long T, long long V, int D, bool dw_f32) {
  Plan pl;
  const long long rows = std::max<long long>(T, 1);
  pl.two = T <= kTwoTermRows;
  pl.g2_rows = pl.two ? kTwoTermRows : dw_f32 ? rows : 0;
  pl.dx_rows = pl.two ? 2 * kTwoTermRows : rows;
  const long long g_rows = (pl.two ? kTwoTermRows : rows) + pl.g2_rows;
  pl.piece = std::max<long long>(1, (long long)(kPieceBytes / 2 / kTN) / g_rows) * kTN;
  pl.piece = std::min(pl.piece, ceil_div<long long>(V, kTN) * kTN);
  pl.pieces = (int)ceil_div<long long>(V, pl.piece);
  pl.ldg = pl.piece;
  dx_ranges(T, D, std::min(pl.piece, V), &pl.dx_splits, &pl.dx_ksteps);
  size_t at = dash::kWsHeaderBytes;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at = round_up_to(at + bytes, 256);
    return here;
  };
  pl.ztgt = take(rows * 4);
  pl.part = take((size_t)2 * ceil_div<long long>(V, kTN) * rows * sizeof(float2));
  const size_t fwd = at;
  at = dash::kWsHeaderBytes;
  pl.g = take((size_t)g_rows * pl.ldg * 2);
  pl.acc = take(pl.pieces > 1 ? (size_t)rows * D * 4 : 0);
  pl.joined = pl.dx_splits > 1 || pl.two;
  pl.dx_part = take(pl.joined ? (size_t)pl.dx_splits * pl.dx_rows * D * 4 : 0);
  pl.total = std::max(fwd, at);
  return pl;
}

// What both directions need, whatever dW's type.
size_t workspace_size(long long T, long long V, int D) {
  return std::max(make_plan(T, V, D, false).total, make_plan(T, V, D, true).total);
}

// Row-major bf16 (or fp32) [rows][cols], `ld` elements between rows; box = 128 bytes of columns x
// box_rows.
bool map_2d(CUtensorMap* m, const void* ptr, long long rows, long long cols, long long ld, int box_rows,
            bool f32 = false) {
  const int e = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * e};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / e), (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return dash::tensor_map_encoder()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims,
                                    strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

dash_status_t check_args(const void* x, const void* w, const void* targets, const void* a, const void* b,
                         void* workspace, size_t workspace_bytes, long long T, long long V, int D,
                         long long ldx, long long ldw, float scale, int id_bits) {
  if (!w || !workspace || (T > 0 && (!x || !targets || !a || !b))) return DASH_ERR_INVALID_ARG;
  if (T < 0 || V < 1 || D < 1 || !(scale > 0.f)) return DASH_ERR_INVALID_ARG;
  if (id_bits != 32 && id_bits != 64) return DASH_ERR_INVALID_ARG;
  if (!sizes_ok(T, V, D)) return DASH_ERR_UNSUPPORTED;
  if (ldx < D || ldw < D) return DASH_ERR_INVALID_ARG;
  if (ldx % 8 || ldw % 8 || ldx > (1ll << 38) || ldw > (1ll << 38)) return DASH_ERR_UNSUPPORTED;
  if (!is_aligned(x, 16) || !is_aligned(w, 16) || !is_aligned(targets, id_bits / 8) ||
      !is_aligned(a, 4) || !is_aligned(b, 4))
    return DASH_ERR_INVALID_ARG;
  if (!is_aligned(workspace, 256)) return DASH_ERR_INVALID_ARG;
  if (workspace_bytes < workspace_size(T, V, D)) return DASH_ERR_WORKSPACE_TOO_SMALL;
  if (!dash::tensor_map_encoder()) {
    dash::set_last_error("cuTensorMapEncodeTiled is not available from the driver");
    return DASH_ERR_CUDA;
  }
  return DASH_OK;
}

// Fills in the tiles of a product and returns its units of work.
long long set_tiles(Params* p) {
  p->tiles_m = ceil_div(p->M, kTM);
  p->tiles_n = ceil_div(p->N, kTN);
  return (long long)p->tiles_m * p->tiles_n * p->splits;
}

template <int OP, bool SEGMENTS = false>
dash_status_t launch(Params p, const Maps& maps, Second<OP> second, int sms, bool first, cudaStream_t stream) {
  long long units = set_tiles(&p);
  if constexpr (OP == BOTH) units += set_tiles(&second.p);
  if (units >= (1ll << 31) - 1024) {
    dash::set_last_error("too many output tiles for one call");
    return DASH_ERR_UNSUPPORTED;
  }
  DASH_TRY(dash::allow_shared((const void*)gemm_kernel<OP, SEGMENTS>, kSmem<OP>));
  const int grid = 2 * (int)std::min<long long>(units, sms / 2);
  if (first) {
    gemm_kernel<OP, SEGMENTS><<<grid, kXentThreads, kSmem<OP>, stream>>>(p, maps, second);
    DASH_TRY(cudaGetLastError());
  } else {
    DASH_TRY(dash::launch_after(gemm_kernel<OP, SEGMENTS>, dim3(grid), kXentThreads, kSmem<OP>, stream, p, maps, second));
  }
  return DASH_OK;
}

dash_status_t bad_map() {
  dash::set_last_error("cuTensorMapEncodeTiled rejected a tensor");
  return DASH_ERR_CUDA;
}

dash_status_t sm_count(int* sms) {
  int dev = 0;
  DASH_TRY(cudaGetDevice(&dev));
  DASH_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return DASH_OK;
}

}  // namespace

extern "C" {

size_t dash_linear_xent_workspace_size(long long T, long long V, int D) {
  return sizes_ok(T, V, D) ? workspace_size(T, V, D) : 0;
}

dash_status_t dash_linear_xent_fwd(const void* x, const void* w, const void* targets, float* loss,
                                   float* lse, void* workspace, size_t workspace_bytes, long long T,
                                   long long V, int D, long long ldx, long long ldw, float scale,
                                   long long ignore_index, int id_bits, cudaStream_t stream) {
  dash_status_t st = check_args(x, w, targets, loss, lse, workspace, workspace_bytes, T, V, D, ldx, ldw,
                                scale, id_bits);
  if (st != DASH_OK) return st;
  int sms = 0;
  st = sm_count(&sms);
  if (st != DASH_OK) return st;
  char* ws = (char*)workspace;
  if (T == 0) {
    DASH_TRY(cudaMemsetAsync(ws, 0, dash::kWsHeaderBytes, stream));
    return DASH_OK;
  }
  const Plan pl = make_plan(T, V, D, false);
  Maps maps = {};
  if (!map_2d(&maps.a, x, T, D, ldx, kCtaM) || !map_2d(&maps.b, w, V, D, ldw, kCtaN)) return bad_map();
  Params p = {};
  p.M = (int)T;
  p.N = (int)V;
  p.K = D;
  p.splits = 1;
  p.ksteps_per_split = ceil_div(D, kTK);
  p.id_bits = id_bits;
  p.targets = targets;
  p.ignore_index = ignore_index;
  p.scale = scale;
  p.scale_log2 = scale * dash::kLog2e;
  p.part = (float2*)(ws + pl.part);
  p.ztgt = (float*)(ws + pl.ztgt);
  p.V = V;
  p.header = (int*)ws;
  p.timeout_ns = dash::sync_timeout_ns();
  p.withhold = dash::sync_withheld();
  DASH_TRY(cudaMemsetAsync(ws, 0, dash::kWsHeaderBytes, stream));
  st = launch<LSE>(p, maps, {}, sms, true, stream);
  if (st != DASH_OK) return st;
  DASH_TRY(dash::launch_after(lse_join_kernel, dim3((unsigned)ceil_div<long long>(T, 32)), 1024, 0, stream, p.part,
                              p.ztgt, 2 * ceil_div((int)V, kTN), (int)T, targets, id_bits, ignore_index, V, loss,
                              lse, p.header));
  return DASH_OK;
}

dash_status_t dash_linear_xent_bwd(const void* x, const void* w, const void* targets,
                                   const float* lse, const float* dloss, void* dx, void* dw,
                                   void* workspace, size_t workspace_bytes, long long T,
                                   long long V, int D, long long ldx, long long ldw, float scale,
                                   long long ignore_index, int id_bits, int dw_dtype,
                                   int accumulate, cudaStream_t stream) {
  if (!dw || (T > 0 && !dx)) return DASH_ERR_INVALID_ARG;
  if (dw_dtype != DASH_BF16 && dw_dtype != DASH_FP32) return DASH_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DASH_ERR_INVALID_ARG;
  if (!is_aligned(dx, 16) || !is_aligned(dw, 16)) return DASH_ERR_INVALID_ARG;
  dash_status_t st = check_args(x, w, targets, lse, dloss, workspace, workspace_bytes, T, V, D, ldx, ldw,
                                scale, id_bits);
  if (st != DASH_OK) return st;
  int sms = 0;
  st = sm_count(&sms);
  if (st != DASH_OK) return st;
  char* ws = (char*)workspace;
  const size_t dw_elt = dw_dtype == DASH_FP32 ? 4 : 2;
  if (T == 0) {
    DASH_TRY(cudaMemsetAsync(ws, 0, dash::kWsHeaderBytes, stream));
    if (!accumulate) DASH_TRY(cudaMemsetAsync(dw, 0, (size_t)V * D * dw_elt, stream));
    return DASH_OK;
  }
  const Plan pl = make_plan(T, V, D, dw_dtype == DASH_FP32);
  __nv_bfloat16* g = (__nv_bfloat16*)(ws + pl.g);
  Params base = {};
  base.id_bits = id_bits;
  base.targets = targets;
  base.ignore_index = ignore_index;
  base.scale = scale;
  base.scale_log2 = scale * dash::kLog2e;
  base.lse = lse;
  base.dloss = dloss;
  base.g = g;
  base.g2 = pl.g2_rows > 0 ? g + pl.g2_rows * pl.ldg : nullptr;
  base.ldg = pl.ldg;
  base.V = V;
  base.header = (int*)ws;
  base.timeout_ns = dash::sync_timeout_ns();
  base.withhold = dash::sync_withheld();
  base.splits = 1;
  base.seg_steps = kSegSteps16;
  base.two = pl.two;
  base.rows = (int)T;
  Maps grad = {}, dxm = {}, dwm = {};
  if (!map_2d(&grad.a, x, T, D, ldx, kCtaM) || !map_2d(&grad.b, w, V, D, ldw, kCtaN) ||
      !map_2d(&dxm.b, w, V, D, ldw, kTK) || !map_2d(&dwm.b, x, T, D, ldx, kTK))
    return bad_map();
  check_targets_kernel<<<1, 1024, 0, stream>>>(
      targets, id_bits, (int)T, ignore_index, V, base.header);
  DASH_TRY(cudaGetLastError());
  for (int i = 0; i < pl.pieces; ++i) {
    const long long v0 = i * pl.piece, vp = std::min(pl.piece, V - v0);
    const bool first = i == 0, last = i == pl.pieces - 1;
    if (!map_2d(&dxm.a, g, T, vp, pl.ldg, kCtaM) || !map_2d(&dwm.a, g, T, vp, pl.ldg, kTK)) return bad_map();
    dxm.a2 = dxm.a;
    dwm.a2 = dwm.a;
    if (base.g2 && (!map_2d(&dxm.a2, base.g2, T, vp, pl.ldg, kCtaM) || !map_2d(&dwm.a2, base.g2, T, vp, pl.ldg, kTK)))
      return bad_map();
    dwm.c = dwm.a;                       // read only where dW is not accumulated
    if (!accumulate &&
        !map_2d(&dwm.c, (char*)dw + (size_t)v0 * D * dw_elt, vp, D, D, 32, dw_dtype == DASH_FP32))
      return bad_map();
    Params p = base;
    p.b_row0 = (int)v0;
    // G of the piece
    p.M = (int)T;
    p.N = (int)vp;
    p.K = D;
    p.ksteps_per_split = ceil_div(D, kTK);
    st = launch<GRAD>(p, grad, {}, sms, false, stream);
    if (st != DASH_OK) return st;
    // dX += G W
    p.N = D;
    p.K = (int)vp;
    p.out = dx;
    p.splits = 1;
    p.ksteps_per_split = ceil_div((int)vp, kTK);
    p.acc = (float*)(ws + pl.acc);
    p.out_mode = first ? (last ? OUT_BF16 : OUT_F32) : (last ? OUT_BF16_ADD : OUT_F32_ADD);
    if (pl.joined) {
      p.M = (int)pl.dx_rows;
      p.ksteps_per_split = pl.dx_ksteps;
      p.splits = ceil_div(ceil_div((int)vp, kTK), pl.dx_ksteps);
      p.out_mode = OUT_PART;
      p.acc = (float*)(ws + pl.dx_part);
    }
    // dW of the piece = G^T X
    Second<BOTH> dwp;
    dwp.maps = dwm;
    Params& d = dwp.p;
    d = base;
    d.M = (int)vp;
    d.N = D;
    d.K = (int)T;
    d.splits = 1;
    if (dw_dtype == DASH_FP32) d.seg_steps = kSegSteps32;
    d.ksteps_per_split = (base.g2 ? 2 : 1) * ceil_div((int)T, kTK);
    d.out = (char*)dw + (size_t)v0 * D * dw_elt;
    d.out_mode = dw_dtype == DASH_FP32 ? (accumulate ? OUT_F32_ADD : OUT_F32)
                                       : (accumulate ? OUT_BF16_ADD : OUT_BF16);
    const bool dx_long = p.ksteps_per_split > p.seg_steps, dw_long = d.ksteps_per_split > d.seg_steps;
    const bool together = !dx_long && !dw_long && set_tiles(&p) + set_tiles(&d) <= kTogetherRounds * (sms / 2);
    st = together  ? launch<BOTH>(p, dxm, dwp, sms, false, stream)
         : dx_long ? launch<DX, true>(p, dxm, {}, sms, false, stream)
                   : launch<DX>(p, dxm, {}, sms, false, stream);
    if (st != DASH_OK) return st;
    if (pl.joined) {
      const size_t n = (size_t)T * D;
      DASH_TRY(dash::launch_after(dx_join_kernel, dim3((unsigned)ceil_div<size_t>(n, 4 * kJoinThreads)),
                                  kJoinThreads, 0, stream, p.acc,
                                  p.splits, n, (size_t)pl.dx_rows * D,
                                  pl.two ? (size_t)kTwoTermRows * D : (size_t)0, (float*)(ws + pl.acc), (int)first,
                                  (int)last, (__nv_bfloat16*)dx));
    }
    if (!together) {
      st = dw_long ? launch<DW, true>(d, dwm, {}, sms, false, stream) : launch<DW>(d, dwm, {}, sms, false, stream);
      if (st != DASH_OK) return st;
    }
  }
  return DASH_OK;
}

}  // extern "C"
