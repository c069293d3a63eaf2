"""Thin Python binding of the training-step operators in libdash_attn (include/dash_train.h).

As in dash_attn.py the functions only check and marshal their arguments; every step runs in
the library's CUDA kernels on torch's current stream of the tensors' device (or `stream`).
Wrong types, shapes or devices raise ValueError before anything is queued, a status other
than DASH_OK raises DashError. With check=True a call that has a workspace waits for the
stream and raises what the device reported (an index out of range); check=False leaves that
to dash_attn_get_status(workspace).
"""

from __future__ import annotations

import ctypes

import torch

from . import dash_attn as _core
from .dash_attn import DASH_ERR_UNSUPPORTED, DashError, dash_attn_get_status

DASH_BF16, DASH_FP16, DASH_FP32 = 0, 1, 2
_DTYPE = {torch.bfloat16: DASH_BF16, torch.float16: DASH_FP16, torch.float32: DASH_FP32}
_ID_BITS = {torch.int32: 32, torch.int64: 64}

_c_int, _c_float, _c_size, _vp, _ll = (ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                                       ctypes.c_void_p, ctypes.c_longlong)

_llp = ctypes.POINTER(_ll)
_c3 = _ll * 3


class _ClipTensor(ctypes.Structure):
    _fields_ = [("grad", _vp), ("out", _vp), ("numel", _ll), ("dtype", _c_int)]


_core._SIGNATURES.update({
    "dash_embed_fwd": (_c_int, [_vp] * 4 + [_ll, _ll, _c_int, _ll, _ll, _c_float, _c_int, _c_int, _vp]),
    "dash_embed_bwd_workspace_size": (_c_size, [_ll, _ll, _c_int]),
    "dash_embed_bwd": (_c_int, [_vp] * 4 + [_c_size, _ll, _ll, _c_int, _ll, _c_float, _ll] + [_c_int] * 4
                       + [_vp]),
    "dash_qk_norm_rope_fwd": (_c_int, [_vp] * 10 + [_c_int] * 6 + [_ll, _llp, _llp, _ll, _c_float]
                              + [_c_int] * 3 + [_vp]),
    "dash_qk_norm_rope_bwd_workspace_size": (_c_size, [_c_int] * 5),
    "dash_qk_norm_rope_bwd": (_c_int, [_vp] * 14 + [_c_size] + [_c_int] * 6 + [_ll, _llp, _llp, _llp, _llp,
                                                                              _ll, _c_float]
                              + [_c_int] * 3 + [_vp]),
    "dash_grad_clip_plan_size": (_c_size, [ctypes.POINTER(_ClipTensor), _c_int]),
    "dash_grad_clip_plan": (_c_int, [ctypes.POINTER(_ClipTensor), _c_int, _vp, _c_size, _vp]),
    "dash_grad_clip": (_c_int, [_vp, _c_float, _vp, _vp]),
    "dash_linear_xent_workspace_size": (_c_size, [_ll, _ll, _c_int]),
    "dash_linear_xent_fwd": (_c_int, [_vp] * 6 + [_c_size, _ll, _ll, _c_int, _ll, _ll, _c_float, _ll,
                                                  _c_int, _vp]),
    "dash_linear_xent_bwd": (_c_int, [_vp] * 8 + [_c_size, _ll, _ll, _c_int, _ll, _ll, _c_float, _ll,
                                                  _c_int, _c_int, _c_int, _vp]),
})


def _raise(status: int, where: str):
    if status:
        raise DashError(status, where)


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _cuda(t, name: str, device=None):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: expected a CUDA tensor")
    _need(device is None or t.device == device, f"{name}: expected a tensor on {device}")


def _rows(t, name: str):
    """A 2-D tensor whose rows are contiguous; returns the elements between rows."""
    _need(t.dim() == 2 and (t.shape[1] == 1 or t.stride(1) == 1),
          f"{name}: expected 2-D rows of contiguous elements")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _index(t, name: str, device):
    _cuda(t, name, device)
    _need(t.dtype in _ID_BITS and t.is_contiguous(), f"{name}: expected contiguous int32 or int64")
    return _ID_BITS[t.dtype]


def _ws(workspace, name: str = "workspace"):
    _need(workspace.is_cuda and workspace.is_contiguous(), f"{name}: expected a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _finish(workspace, stream, check: bool, where: str):
    if check:
        _raise(dash_attn_get_status(workspace, stream), where + " (device status)")


# ---- token embedding --------------------------------------------------------------------------

def embed_forward(table, ids, scale: float = 1.0, out=None, status=None, stream=None):
    """out[...] = scale * table[ids[...]].

    table: [V, D] bf16, fp16 or fp32 with contiguous rows; ids: contiguous int32 or int64 of
    any shape. status: an optional int32 CUDA tensor of one element, which reads
    DASH_ERR_BOUNDS when an id was out of range (its row is NaN). Returns [*ids.shape, D]."""
    _cuda(table, "table")
    _need(table.dtype in _DTYPE, "table: expected bfloat16, float16 or float32")
    ld = _rows(table, "table")
    bits = _index(ids, "ids", table.device)
    V, D = table.shape
    if out is None:
        out = torch.empty(*ids.shape, D, dtype=table.dtype, device=table.device)
    else:
        _cuda(out, "out", table.device)
        _need(out.dtype == table.dtype and tuple(out.shape) == (*ids.shape, D) and out.is_contiguous(),
              "out: expected contiguous [*ids.shape, D] of the table's type")
    if status is not None:
        _cuda(status, "status", table.device)
        _need(status.dtype == torch.int32 and status.numel() == 1, "status: expected one int32")
    _raise(_core.load().dash_embed_fwd(
        table.data_ptr(), ids.data_ptr(), out.data_ptr(), None if status is None else status.data_ptr(),
        ids.numel(), V, D, ld, D, scale, _DTYPE[table.dtype], bits, _core._stream(table, stream)),
        "dash_embed_fwd")
    return out


def dash_embed_bwd_workspace_size(T: int, V: int, D: int) -> int:
    return int(_core.load().dash_embed_bwd_workspace_size(int(T), int(V), int(D)))


def new_embed_workspace(T: int, V: int, D: int, device) -> torch.Tensor:
    """The workspace of embed_backward for T tokens (uint8)."""
    nbytes = dash_embed_bwd_workspace_size(T, V, D)
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_embed_bwd_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def embed_backward(dout, ids, vocab: int, scale: float = 1.0, padding_idx=None, dtable=None,
                   accumulate: bool = False, workspace=None, stream=None, check: bool = True):
    """Gradient of the table: scale times the sum of dout's rows of each id, in token order.

    dout: [*ids.shape, D] (2-D: rows may be strided); ids as in embed_forward. padding_idx:
    an id whose tokens are left out. dtable: an optional contiguous [vocab, D] tensor of
    dout's type or fp32 to write to, or to add to with accumulate=True. Returns dtable."""
    _cuda(dout, "dout")
    _need(dout.dtype in _DTYPE, "dout: expected bfloat16, float16 or float32")
    bits = _index(ids, "ids", dout.device)
    _need(dout.dim() >= 1 and tuple(dout.shape[:-1]) == tuple(ids.shape), "dout: expected [*ids.shape, D]")
    T, D = ids.numel(), dout.shape[-1]
    if dout.dim() == 2:
        ld = _rows(dout, "dout")
    else:
        _need(dout.is_contiguous(), "dout: expected contiguous")
        ld = D
    if dtable is None:
        _need(not accumulate, "accumulate: needs dtable")
        dtable = torch.empty((vocab, D), dtype=dout.dtype, device=dout.device)
    else:
        _cuda(dtable, "dtable", dout.device)
        _need(dtable.dtype in (dout.dtype, torch.float32) and tuple(dtable.shape) == (vocab, D)
              and dtable.is_contiguous(), "dtable: expected contiguous [vocab, D] of dout's type or float32")
    _need(padding_idx is None or 0 <= padding_idx < vocab, "padding_idx: out of range")
    if workspace is None:
        workspace = new_embed_workspace(T, vocab, D, dout.device)
    ws, nbytes = _ws(workspace)
    _raise(_core.load().dash_embed_bwd(
        dout.data_ptr(), ids.data_ptr(), dtable.data_ptr(), ws, nbytes, T, vocab, D, ld, scale,
        -1 if padding_idx is None else padding_idx, int(accumulate), _DTYPE[dout.dtype],
        _DTYPE[dtable.dtype], bits, _core._stream(dout, stream)), "dash_embed_bwd")
    _finish(workspace, stream, check, "dash_embed_bwd")
    return dtable


# ---- norm and rotation of queries and keys ----------------------------------------------------

def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, device="cuda"):
    """(cos, sin), fp32 [positions, rotary_dim / 2]: angle p base^(-2i / rotary_dim), computed
    in 64 bits, where 32 would lose the far positions' angles."""
    inv = torch.pow(float(base), -torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64) / rotary_dim)
    ang = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _heads(t, name: str, like=None):
    """[B, S, H, D] with contiguous D; returns its {batch, token, head} strides. Strides of
    dimensions of one element are never used and count as zero."""
    _need(t.dim() == 4 and (t.shape[3] == 1 or t.stride(3) == 1), f"{name}: expected [B, S, H, D], D contiguous")
    if like is not None:
        _need(t.dtype == like.dtype and t.device == like.device and t.shape[:2] == like.shape[:2]
              and t.shape[3] == like.shape[3], f"{name}: expected the type, device and [B, S, ., D] of q")
    n, st = t.shape, t.stride()
    return _c3(st[0] if n[0] > 1 else 0, st[1] if n[1] > 1 else 0, st[2] if n[2] > 1 else 0)


def _qk_args(q, k, wq, wk, cos, sin, positions):
    _cuda(q, "q")
    _cuda(k, "k", q.device)
    _need(q.dtype in _DTYPE, "q: expected bfloat16, float16 or float32")
    qs, ks = _heads(q, "q"), _heads(k, "k", q)
    B, S, Hq, D = q.shape
    for w, name in ((wq, "wq"), (wk, "wk")):
        if w is not None:
            _cuda(w, name, q.device)
            _need(w.dtype == torch.float32 and tuple(w.shape) == (D,) and w.is_contiguous(),
                  f"{name}: expected contiguous float32 [D]")
    _cuda(cos, "cos", q.device)
    _cuda(sin, "sin", q.device)
    _need(cos.dtype == torch.float32 and sin.dtype == torch.float32 and cos.dim() == 2
          and cos.shape == sin.shape and cos.is_contiguous() and sin.is_contiguous(),
          "cos and sin: expected contiguous float32 [P, R / 2]")
    P, R = cos.shape[0], 2 * cos.shape[1]
    pos, stride, bits = None, 0, 32
    if positions is not None:
        bits = _index(positions, "positions", q.device)
        _need(tuple(positions.shape) in ((B, S), (S,), (1, S)), "positions: expected [B, S] or [S]")
        pos, stride = positions.data_ptr(), S if positions.dim() == 2 and positions.shape[0] == B else 0
    return qs, ks, B, S, Hq, k.shape[2], D, R, P, pos, stride, bits


def _ptr(t):
    return None if t is None else t.data_ptr()


def qk_norm_rope_forward(q, k, wq, wk, cos, sin, positions=None, eps: float = 1e-6, interleaved: bool = False,
                         status=None, stream=None):
    """Norm over each head's D values (times wq, wk), then the rotation, of queries and keys.

    q: [B, S, Hq, D], k: [B, S, Hk, D], bf16, fp16 or fp32, D contiguous, any strides that are
    multiples of 8 (parts of a fused projection, transposed [B, H, S, D]); wq, wk: fp32 [D] or
    None; cos, sin: fp32 [P, R / 2] (rope_table); positions: int [B, S] or [S], default 0 .. S - 1;
    interleaved: pairs (2i, 2i + 1) rather than (i, i + R / 2). status as in embed_forward.
    Returns contiguous (q_out, k_out) as attn_forward takes them."""
    qs, ks, B, S, Hq, Hk, D, R, P, pos, stride, bits = _qk_args(q, k, wq, wk, cos, sin, positions)
    q_out = torch.empty((B, S, Hq, D), dtype=q.dtype, device=q.device)
    k_out = torch.empty((B, S, Hk, D), dtype=q.dtype, device=q.device)
    if status is not None:
        _cuda(status, "status", q.device)
        _need(status.dtype == torch.int32 and status.numel() == 1, "status: expected one int32")
    _raise(_core.load().dash_qk_norm_rope_fwd(
        q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), cos.data_ptr(), sin.data_ptr(), pos,
        q_out.data_ptr(), k_out.data_ptr(), _ptr(status), B, S, Hq, Hk, D, R, P, qs, ks, stride, eps,
        int(interleaved), _DTYPE[q.dtype], bits, _core._stream(q, stream)), "dash_qk_norm_rope_fwd")
    return q_out, k_out


def dash_qk_norm_rope_bwd_workspace_size(B: int, S: int, Hq: int, Hk: int, D: int) -> int:
    return int(_core.load().dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D))


def new_qk_norm_rope_workspace(B: int, S: int, Hq: int, Hk: int, D: int, device) -> torch.Tensor:
    """The workspace of qk_norm_rope_backward (uint8)."""
    nbytes = dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D)
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_qk_norm_rope_bwd_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None,
                          check: bool = True):
    """Gradients of qk_norm_rope_forward with respect to q, k, wq and wk.

    dq_out, dk_out: contiguous, as attn_backward returns them. dq, dk: optional tensors to
    write to, strided like q and k may be (parts of a fused projection's gradient). Returns
    (dq, dk, dwq, dwk), the last two fp32 [D] or None where the weight is None."""
    qs, ks, B, S, Hq, Hk, D, R, P, pos, stride, bits = _qk_args(q, k, wq, wk, cos, sin, positions)
    for t, like, name in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")):
        _cuda(t, name, q.device)
        _need(t.dtype == q.dtype and t.shape == like.shape and t.is_contiguous(),
              f"{name}: expected contiguous, of the input's type and shape")
    if dq is None:
        dq = torch.empty((B, S, Hq, D), dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty((B, S, Hk, D), dtype=q.dtype, device=q.device)
    for t, like, name in ((dq, q, "dq"), (dk, k, "dk")):
        _cuda(t, name, q.device)
        _need(t.dtype == q.dtype and t.shape == like.shape, f"{name}: expected the input's type and shape")
    dqs, dks = _heads(dq, "dq"), _heads(dk, "dk")
    dwq = None if wq is None else torch.empty(D, dtype=torch.float32, device=q.device)
    dwk = None if wk is None else torch.empty(D, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_qk_norm_rope_workspace(B, S, Hq, Hk, D, q.device)
    ws, nbytes = _ws(workspace)
    _raise(_core.load().dash_qk_norm_rope_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk),
        cos.data_ptr(), sin.data_ptr(), pos, dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk), ws, nbytes,
        B, S, Hq, Hk, D, R, P, qs, ks, dqs, dks, stride, eps, int(interleaved), _DTYPE[q.dtype], bits,
        _core._stream(q, stream)), "dash_qk_norm_rope_bwd")
    _finish(workspace, stream, check, "dash_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ---- gradient norm and clipping -----------------------------------------------------------------

class GradClipPlan:
    """The tensors of grad_clip and their table on the device. Holds the tensors, so that the
    addresses in the table stay theirs; build a new plan when a gradient is replaced."""

    def __init__(self, grads, outs, table, norm):
        self.grads, self.outs, self.table, self.norm = grads, outs, table, norm


def grad_clip_plan(grads, out=None, stream=None) -> GradClipPlan:
    """Plan of clipping `grads` (contiguous bf16, fp16 or fp32 CUDA tensors of one device, which
    overlap one another nowhere) in place, or into the tensors `out` of the same shapes and
    types."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    _need(len(grads) > 0 and len(outs) == len(grads), "grads: expected tensors, as many as out")
    dev = grads[0].device
    arr = (_ClipTensor * len(grads))()
    spans = set()
    for i, (g, o) in enumerate(zip(grads, outs)):
        for t, name in ((g, "grads"), (o, "out")):
            _cuda(t, f"{name}[{i}]", dev)
            _need(t.dtype in _DTYPE and t.is_contiguous(),
                  f"{name}[{i}]: expected contiguous bfloat16, float16 or float32")
            if t.numel():
                spans.add((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i))
        _need(o.dtype == g.dtype and o.shape == g.shape, f"out[{i}]: expected the type and shape of grads[{i}]")
        arr[i] = _ClipTensor(g.data_ptr(), o.data_ptr(), g.numel(), _DTYPE[g.dtype])
    spans = sorted(spans)
    _need(all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), "grads and out: tensors overlap")
    lib = _core.load()
    nbytes = lib.dash_grad_clip_plan_size(arr, len(grads))
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_grad_clip_plan_size")
    table = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _raise(lib.dash_grad_clip_plan(arr, len(grads), table.data_ptr(), nbytes, _core._stream(table, stream)),
           "dash_grad_clip_plan")
    return GradClipPlan(grads, outs, table, torch.empty((), dtype=torch.float32, device=dev))


def grad_clip(plan: GradClipPlan, max_norm: float, stream=None):
    """Global L2 norm of the plan's gradients, which are scaled by max_norm / norm when it is
    above max_norm. Returns (norm, tensors): norm is a device fp32 scalar that the next call
    overwrites."""
    _raise(_core.load().dash_grad_clip(plan.table.data_ptr(), max_norm, plan.norm.data_ptr(),
                                       _core._stream(plan.table, stream)), "dash_grad_clip")
    return plan.norm, plan.outs


# ---- cross entropy from hidden states -------------------------------------------------------

def dash_linear_xent_workspace_size(T: int, V: int, D: int) -> int:
    return int(_core.load().dash_linear_xent_workspace_size(int(T), int(V), int(D)))


def new_linear_xent_workspace(T: int, V: int, D: int, device) -> torch.Tensor:
    """The workspace of linear_xent_forward and _backward for these sizes (uint8)."""
    nbytes = dash_linear_xent_workspace_size(T, V, D)
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_linear_xent_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _xent_args(x, w, targets):
    _cuda(x, "x")
    _cuda(w, "w", x.device)
    _need(x.dtype == torch.bfloat16 and w.dtype == torch.bfloat16, "x and w: expected bfloat16")
    ldx, ldw = _rows(x, "x"), _rows(w, "w")
    bits = _index(targets, "targets", x.device)
    T, D = x.shape
    _need(w.shape[1] == D, "w: expected as many columns as x")
    _need(targets.dim() == 1 and targets.shape[0] == T, "targets: expected one index a row of x")
    return T, w.shape[0], D, ldx, ldw, bits


def linear_xent_forward(x, w, targets, ignore_index: int = -100, scale: float = 1.0, workspace=None,
                        stream=None, check: bool = True):
    """Softmax cross entropy of the logits scale * x w^T, which are never stored.

    x: bf16 [T, D] hidden states, w: bf16 [V, D] output embedding, targets: int [T].
    Returns (loss, lse), fp32 [T]; rows whose target is ignore_index have loss 0."""
    T, V, D, ldx, ldw, bits = _xent_args(x, w, targets)
    if workspace is None:
        workspace = new_linear_xent_workspace(T, V, D, x.device)
    out = torch.empty((2, T), dtype=torch.float32, device=x.device)
    loss, lse = out[0], out[1]
    ws, nbytes = _ws(workspace)
    _raise(_core.load().dash_linear_xent_fwd(
        x.data_ptr(), w.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(), ws, nbytes,
        T, V, D, ldx, ldw, scale, ignore_index, bits, _core._stream(x, stream)), "dash_linear_xent_fwd")
    _finish(workspace, stream, check, "dash_linear_xent_fwd")
    return loss, lse


def linear_xent_backward(x, w, targets, lse, dloss, ignore_index: int = -100, scale: float = 1.0,
                         dw=None, accumulate: bool = False, dw_dtype=None, workspace=None, stream=None,
                         check: bool = True):
    """Gradients of sum(dloss * loss) with respect to x (bf16 [T, D]) and w.

    lse: from linear_xent_forward; dloss: fp32 [T]. dw: an optional [V, D] bf16 or fp32
    tensor to write to, or to add to with accumulate=True (tied embeddings, several
    micro-batches); else one of dw_dtype (bf16) is allocated. Returns (dx, dw)."""
    T, V, D, ldx, ldw, bits = _xent_args(x, w, targets)
    for t, name in ((lse, "lse"), (dloss, "dloss")):
        _cuda(t, name, x.device)
        _need(t.dtype == torch.float32 and tuple(t.shape) == (T,) and t.is_contiguous(),
              f"{name}: expected contiguous float32 [T]")
    if dw is None:
        _need(not accumulate, "accumulate: needs dw")
        dw = torch.empty((V, D), dtype=dw_dtype or torch.bfloat16, device=x.device)
    _cuda(dw, "dw", x.device)
    _need(dw.dtype in (torch.bfloat16, torch.float32) and tuple(dw.shape) == (V, D) and dw.is_contiguous(),
          "dw: expected contiguous bfloat16 or float32 [V, D]")
    if workspace is None:
        workspace = new_linear_xent_workspace(T, V, D, x.device)
    dx = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    ws, nbytes = _ws(workspace)
    _raise(_core.load().dash_linear_xent_bwd(
        x.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(), dloss.data_ptr(), dx.data_ptr(),
        dw.data_ptr(), ws, nbytes, T, V, D, ldx, ldw, scale, ignore_index, bits, _DTYPE[dw.dtype],
        int(accumulate), _core._stream(x, stream)), "dash_linear_xent_bwd")
    _finish(workspace, stream, check, "dash_linear_xent_bwd")
    return dx, dw
