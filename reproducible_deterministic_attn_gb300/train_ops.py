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

_core._SIGNATURES.update({
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
