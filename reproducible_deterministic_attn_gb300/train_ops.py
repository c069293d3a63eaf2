"""Thin Python binding of the training-step operators in libdash_attn (include/dash_train.h).

As in dash_attn.py the functions only check and marshal their arguments; every step runs in
the library's CUDA kernels on torch's current stream of the tensors' device, which a call makes
the current one for its time (or on `stream`, a stream of that device, on which it then also
allocates what it returns and uses).
Wrong types, shapes or devices raise ValueError before anything is queued, a status other
than DASH_OK raises DashError. With check=True a call that has a workspace waits for the
stream and raises what the device reported (an index out of range); check=False leaves that
to dash_attn_get_status(workspace).
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import dash_attn as _core
from .dash_attn import DASH_ERR_UNSUPPORTED, DashError, dash_attn_get_status

DASH_BF16, DASH_FP16, DASH_FP32 = 0, 1, 2
_DTYPE = {torch.bfloat16: DASH_BF16, torch.float16: DASH_FP16, torch.float32: DASH_FP32}
_ID_BITS = {torch.int32: 32, torch.int64: 64}
_F32, _BF16 = torch.float32, torch.bfloat16

_c_int, _c_float, _c_size, _vp, _ll = (ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                                       ctypes.c_void_p, ctypes.c_longlong)

_c3 = _ll * 3
_c2 = _ll * 2
_ACT = {None: 0, "none": 0, "silu": 1}


class _ClipTensor(ctypes.Structure):
    _fields_ = [("grad", _vp), ("out", _vp), ("numel", _ll), ("dtype", _c_int)]


_core._SIGNATURES.update({
    "dash_embed_fwd": (_c_int, [_vp] * 4 + [_ll, _ll, _c_int, _ll, _ll, _c_float, _c_int, _c_int, _vp]),
    "dash_embed_bwd_workspace_size": (_c_size, [_ll, _ll, _c_int]),
    "dash_embed_bwd": (_c_int, [_vp] * 4 + [_c_size, _ll, _ll, _c_int, _ll, _c_float, _ll] + [_c_int] * 4
                       + [_vp]),
    "dash_qk_norm_rope_fwd": (_c_int, [_vp] * 10 + [_c_int] * 6 + [_ll, _vp, _vp, _ll, _c_float]
                              + [_c_int] * 3 + [_vp]),
    "dash_qk_norm_rope_bwd_workspace_size": (_c_size, [_c_int] * 5),
    "dash_qk_norm_rope_bwd": (_c_int, [_vp] * 14 + [_c_size] + [_c_int] * 6 + [_ll] + [_vp] * 4 + [_ll, _c_float]
                              + [_c_int] * 3 + [_vp]),
    "dash_qk_norm_rope_axes_fwd": (_c_int, [_vp] * 10 + [_c_int] * 6 + [_ll, _vp, _vp, _vp, _c_int, _ll, _ll, _c_float]
                                   + [_c_int] * 3 + [_vp]),
    "dash_qk_norm_rope_axes_bwd": (_c_int, [_vp] * 14 + [_c_size] + [_c_int] * 6 + [_ll] + [_vp] * 5
                                   + [_c_int, _ll, _ll, _c_float] + [_c_int] * 3 + [_vp]),
    "dash_grad_clip_plan_size": (_c_size, [ctypes.POINTER(_ClipTensor), _c_int]),
    "dash_grad_clip_plan": (_c_int, [ctypes.POINTER(_ClipTensor), _c_int, _vp, _c_size, _vp]),
    "dash_grad_clip": (_c_int, [_vp, _c_size, _c_float, _vp, _vp]),
    "dash_linear_xent_workspace_size": (_c_size, [_ll, _ll, _c_int]),
    "dash_linear_xent_fwd": (_c_int, [_vp] * 6 + [_c_size, _ll, _ll, _c_int, _ll, _ll, _c_float, _ll,
                                                  _c_int, _vp]),
    "dash_linear_xent_bwd": (_c_int, [_vp] * 8 + [_c_size, _ll, _ll, _c_int, _ll, _ll, _c_float, _ll,
                                                  _c_int, _c_int, _c_int, _vp]),
    "dash_group_norm_workspace_size": (_c_size, [_ll, _ll, _ll, _c_int]),
    "dash_group_norm_fwd": (_c_int, [_vp] * 7 + [_c_size, _ll, _ll, _ll, _c_int, _vp, _c_float, _c_int, _c_int, _vp]),
    "dash_group_norm_bwd": (_c_int, [_vp] * 10 + [_c_size, _ll, _ll, _ll, _c_int, _vp, _c_int, _c_int, _vp]),
    "dash_cross_attn_fwd_workspace_size": (_c_size, [_c_int] * 6),
    "dash_cross_attn_fwd": (_c_int, [_vp] * 8 + [_c_size] + [_c_int] * 6 + [_vp] * 3 + [_c_float, _c_int, _vp]),
    "dash_cross_attn_bwd_workspace_size": (_c_size, [_c_int] * 6),
    "dash_cross_attn_bwd": (_c_int, [_vp] * 11 + [_c_size] + [_c_int] * 6 + [_vp] * 6 + [_c_float, _c_int, _vp]),
})


# The checks below run on every call, next to kernels of a few microseconds: conditions first,
# messages only once one has failed. A device is its index, -1 for the host.

def _raise(status: int, where: str):
    if status:
        raise DashError(status, where)


def _bad(what: str):
    raise ValueError(what)


def _device(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        _bad(f"{name}: expected a CUDA tensor")
    return dev


def _on(t, name: str, dev: int):
    if t.get_device() != dev:
        _bad(f"{name}: expected a tensor on cuda:{dev}")


def _stream(dev: int) -> int:
    """The raw handle of torch's current stream on the device."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _using(stream, t):
    """Makes `stream` (a torch stream or a raw handle) the current one, so that what a call
    allocates belongs to the stream that its kernels run on."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
        stream = (torch.cuda.ExternalStream(handle, device=t.device) if handle
                  else torch.cuda.default_stream(t.device))
    if stream.device.index != t.get_device():
        _bad(f"stream: expected a stream of the tensors' device, {t.device}")
    return torch.cuda.stream(stream)


def _rows(t, name: str):
    """A 2-D tensor whose rows are contiguous: its sizes and the elements between rows."""
    if t.dim() != 2:
        _bad(f"{name}: expected two dimensions")
    n, d = t.shape
    ld, one = t.stride()
    if one != 1 and d > 1:
        _bad(f"{name}: expected rows of contiguous elements")
    return n, d, ld if n > 1 else max(d, 1)


def _index(t, name: str, dev: int):
    bits = _ID_BITS.get(t.dtype)
    if bits is None or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name}: expected contiguous int32 or int64 on cuda:{dev}")
    return bits


def _vector(t, name: str, n: int, dev: int):
    """A contiguous fp32 [n] tensor's address."""
    if t.dtype != _F32 or t.get_device() != dev or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        _bad(f"{name}: expected contiguous float32 [{n}] on cuda:{dev}")
    return t.data_ptr()


def _status_word(t, dev: int):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != 1 or t.get_device() != dev:
        _bad(f"status: expected one int32 on cuda:{dev}")
    return t.data_ptr()


def _ws(t, dev: int):
    if t.get_device() != dev or not t.is_contiguous():
        _bad(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.nbytes


def _finish(workspace, check: bool, where: str):
    if check:
        _raise(dash_attn_get_status(workspace), where + " (device status)")


# ---- token embedding --------------------------------------------------------------------------

def embed_forward(table, ids, scale: float = 1.0, out=None, status=None, stream=None):
    """out[...] = scale * table[ids[...]].

    table: [V, D] bf16, fp16 or fp32 with contiguous rows; ids: contiguous int32 or int64 of
    any shape. status: an optional int32 CUDA tensor of one element, which reads
    DASH_ERR_BOUNDS when an id was out of range (its row is NaN). Returns [*ids.shape, D]."""
    if stream is not None:
        with _using(stream, table):
            return embed_forward(table, ids, scale, out, status)
    dev = _device(table, "table")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return embed_forward(table, ids, scale, out, status)
    dtype = _DTYPE.get(table.dtype)
    if dtype is None:
        _bad("table: expected bfloat16, float16 or float32")
    V, D, ld = _rows(table, "table")
    bits = _index(ids, "ids", dev)
    if out is None:
        out = table.new_empty((*ids.shape, D))
    elif (out.dtype != table.dtype or out.shape != (*ids.shape, D) or not out.is_contiguous()
          or out.get_device() != dev):
        _bad(f"out: expected contiguous [*ids.shape, D] of the table's type on cuda:{dev}")
    _raise(_core.load().dash_embed_fwd(
        table.data_ptr(), ids.data_ptr(), out.data_ptr(), _status_word(status, dev), ids.numel(), V, D, ld, D,
        scale, dtype, bits, _stream(dev)), "dash_embed_fwd")
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
    if stream is not None:
        with _using(stream, dout):
            return embed_backward(dout, ids, vocab, scale, padding_idx, dtable, accumulate, workspace, check=check)
    dev = _device(dout, "dout")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return embed_backward(dout, ids, vocab, scale, padding_idx, dtable, accumulate, workspace, check=check)
    dtype = _DTYPE.get(dout.dtype)
    if dtype is None:
        _bad("dout: expected bfloat16, float16 or float32")
    bits = _index(ids, "ids", dev)
    shape = dout.shape
    if not shape or shape[:-1] != ids.shape:
        _bad("dout: expected [*ids.shape, D]")
    T, D = ids.numel(), shape[-1]
    if len(shape) == 2:
        ld = _rows(dout, "dout")[2]
    else:
        if not dout.is_contiguous():
            _bad("dout: expected contiguous")
        ld = max(D, 1)
    if dtable is None:
        if accumulate:
            _bad("accumulate: needs dtable")
        dtable = dout.new_empty((vocab, D))
    elif (dtable.dtype not in (dout.dtype, _F32) or dtable.shape != (vocab, D) or not dtable.is_contiguous()
          or dtable.get_device() != dev):
        _bad(f"dtable: expected contiguous [vocab, D] of dout's type or float32 on cuda:{dev}")
    if padding_idx is None:
        padding_idx = -1
    elif not 0 <= padding_idx < vocab:
        _bad("padding_idx: out of range")
    if workspace is None:
        workspace = new_embed_workspace(T, vocab, D, dout.device)
    ws, nbytes = _ws(workspace, dev)
    _raise(_core.load().dash_embed_bwd(
        dout.data_ptr(), ids.data_ptr(), dtable.data_ptr(), ws, nbytes, T, vocab, D, ld, scale, padding_idx,
        accumulate, dtype, _DTYPE[dtable.dtype], bits, _stream(dev)), "dash_embed_bwd")
    _finish(workspace, check, "dash_embed_bwd")
    return dtable


# ---- norm and rotation of queries and keys ----------------------------------------------------

def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, device="cuda"):
    """(cos, sin), fp32 [positions, rotary_dim / 2]: angle p base^(-2i / rotary_dim), computed
    in 64 bits, where 32 would lose the far positions' angles."""
    inv = torch.pow(float(base), -torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64) / rotary_dim)
    ang = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


@functools.lru_cache(maxsize=1024)
def _strides(batch: int, token: int, head: int):
    """Three strides as the C calls read them: the array, which the caller holds for the time
    of its call, and its address."""
    arr = _c3(batch, token, head)
    return arr, ctypes.addressof(arr)


def _heads(t, name: str, dtype, dev: int):
    """[B, S, H, D] with contiguous D: its sizes and its {batch, token, head} strides. Strides of
    dimensions of one element are never used and count as zero."""
    if t.dtype != dtype or t.get_device() != dev or t.dim() != 4:
        _bad(f"{name}: expected [B, S, H, D] of type {dtype} on cuda:{dev}")
    B, S, H, D = t.shape
    sb, ss, sh, one = t.stride()
    if one != 1 and D > 1:
        _bad(f"{name}: expected D contiguous")
    return B, S, H, D, _strides(sb if B > 1 else 0, ss if S > 1 else 0, sh if H > 1 else 0)


def _qk_args(q, k, wq, wk, cos, sin, positions):
    dev = _device(q, "q")
    dtype = q.dtype
    if dtype not in _DTYPE:
        _bad("q: expected bfloat16, float16 or float32")
    B, S, Hq, D, qs = _heads(q, "q", dtype, dev)
    Bk, Sk, Hk, Dk, ks = _heads(k, "k", dtype, dev)
    if Bk != B or Sk != S or Dk != D:
        _bad("k: expected the [B, S, ., D] of q")
    pwq = None if wq is None else _vector(wq, "wq", D, dev)
    pwk = None if wk is None else _vector(wk, "wk", D, dev)
    if (cos.dtype != _F32 or sin.dtype != _F32 or cos.dim() != 2 or cos.shape != sin.shape
            or not cos.is_contiguous() or not sin.is_contiguous() or cos.get_device() != dev
            or sin.get_device() != dev):
        _bad(f"cos and sin: expected contiguous float32 [P, R / 2] on cuda:{dev}")
    P, half = cos.shape
    pos, stride, bits = None, 0, 32
    if positions is not None:
        bits = _index(positions, "positions", dev)
        shape = positions.shape
        if shape == (B, S):
            stride = S
        elif shape != (S,) and shape != (1, S):
            _bad("positions: expected [B, S] or [S]")
        pos = positions.data_ptr()
    return dev, (pwq, pwk, cos.data_ptr(), sin.data_ptr(), pos), (B, S, Hq, Hk, D, 2 * half, P, qs[1], ks[1]), \
        stride, bits, (qs, ks)


def qk_norm_rope_forward(q, k, wq, wk, cos, sin, positions=None, eps: float = 1e-6, interleaved: bool = False,
                         status=None, stream=None):
    """Norm over each head's D values (times wq, wk), then the rotation, of queries and keys.

    q: [B, S, Hq, D], k: [B, S, Hk, D], bf16, fp16 or fp32, D contiguous, any strides that are
    multiples of 8 (parts of a fused projection, transposed [B, H, S, D]); wq, wk: fp32 [D] or
    None; cos, sin: fp32 [P, R / 2] (rope_table); positions: int [B, S] or [S], default 0 .. S - 1;
    interleaved: pairs (2i, 2i + 1) rather than (i, i + R / 2). status as in embed_forward.
    Returns contiguous (q_out, k_out) as attn_forward takes them."""
    if stream is not None:
        with _using(stream, q):
            return qk_norm_rope_forward(q, k, wq, wk, cos, sin, positions, eps, interleaved, status)
    dev, tables, sizes, stride, bits, held = _qk_args(q, k, wq, wk, cos, sin, positions)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return qk_norm_rope_forward(q, k, wq, wk, cos, sin, positions, eps, interleaved, status)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _raise(_core.load().dash_qk_norm_rope_fwd(
        q.data_ptr(), k.data_ptr(), *tables, q_out.data_ptr(), k_out.data_ptr(), _status_word(status, dev),
        *sizes, stride, eps, interleaved, _DTYPE[q.dtype], bits, _stream(dev)), "dash_qk_norm_rope_fwd")
    return q_out, k_out


def dash_qk_norm_rope_bwd_workspace_size(B: int, S: int, Hq: int, Hk: int, D: int) -> int:
    return int(_core.load().dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D))


def new_qk_norm_rope_workspace(B: int, S: int, Hq: int, Hk: int, D: int, device) -> torch.Tensor:
    """The workspace of qk_norm_rope_backward (uint8)."""
    nbytes = dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D)
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_qk_norm_rope_bwd_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _qk_grads(dq_out, dk_out, q, k, wq, wk, sizes, dq, dk, workspace, dev):
    """What the gradients' calls write: (dq, dk, dwq, dwk), the addresses of these and of the
    workspace, the strides of dq and dk, and the workspace."""
    dtype, qshape, kshape, D = q.dtype, q.shape, k.shape, sizes[4]
    if (dq_out.dtype != dtype or dq_out.shape != qshape or not dq_out.is_contiguous() or dq_out.get_device() != dev
            or dk_out.dtype != dtype or dk_out.shape != kshape or not dk_out.is_contiguous()
            or dk_out.get_device() != dev):
        _bad(f"dq_out and dk_out: expected contiguous, of the type and shape of q and k, on cuda:{dev}")
    if dq is None:
        dq = torch.empty(qshape, dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty(kshape, dtype=k.dtype, device=k.device)
    dqn, dkn = _heads(dq, "dq", dtype, dev), _heads(dk, "dk", dtype, dev)
    if dqn[:4] != qshape or dkn[:4] != kshape:
        _bad("dq and dk: expected the shapes of q and k")
    dwq = pdwq = dwk = pdwk = None
    if wq is not None:
        dwq = torch.empty(D, dtype=_F32, device=q.device)
        pdwq = dwq.data_ptr()
    if wk is not None:
        dwk = torch.empty(D, dtype=_F32, device=q.device)
        pdwk = dwk.data_ptr()
    if workspace is None:
        workspace = new_qk_norm_rope_workspace(*sizes[:5], q.device)
    return dq, dk, dwq, dwk, (dq.data_ptr(), dk.data_ptr(), pdwq, pdwk, *_ws(workspace, dev)), (dqn[4], dkn[4]), workspace


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None,
                          check: bool = True):
    """Gradients of qk_norm_rope_forward with respect to q, k, wq and wk.

    dq_out, dk_out: contiguous, as attn_backward returns them. dq, dk: optional tensors to
    write to, strided like q and k may be (parts of a fused projection's gradient). Returns
    (dq, dk, dwq, dwk), the last two fp32 [D] or None where the weight is None."""
    if stream is not None:
        with _using(stream, q):
            return qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, eps, interleaved, dq,
                                         dk, workspace, check=check)
    dev, tables, sizes, stride, bits, held = _qk_args(q, k, wq, wk, cos, sin, positions)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, eps, interleaved, dq,
                                         dk, workspace, check=check)
    dq, dk, dwq, dwk, ptrs, outs, workspace = _qk_grads(dq_out, dk_out, q, k, wq, wk, sizes, dq, dk, workspace, dev)
    _raise(_core.load().dash_qk_norm_rope_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), *tables, *ptrs, *sizes, outs[0][1],
        outs[1][1], stride, eps, interleaved, _DTYPE[q.dtype], bits, _stream(dev)), "dash_qk_norm_rope_bwd")
    _finish(workspace, check, "dash_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def rope_axes_table(positions: int, sections, base: float = 10000.0, own_ladders: bool = False, device="cuda"):
    """(cos, sin), fp32 [positions, sum(sections)], for qk_norm_rope_axes_forward: one ladder of
    frequencies over all pairs (base^(-i / pairs) for pair i), or with own_ladders one for each
    section, which starts anew at 1."""
    sections = [int(n) for n in sections]
    if own_ladders:
        exps = [torch.arange(n, device=device, dtype=torch.float64) / max(n, 1) for n in sections]
        exps = torch.cat(exps) if exps else torch.empty(0, device=device, dtype=torch.float64)
    else:
        exps = torch.arange(sum(sections), device=device, dtype=torch.float64) / max(sum(sections), 1)
    ang = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * torch.pow(float(base), -exps)
    return ang.cos().float(), ang.sin().float()


@functools.lru_cache(maxsize=1024)
def _sections(sections: tuple):
    """Section lengths as the C calls read them: the array, which the caller holds for the time of
    its call, and its address."""
    arr = (_c_int * max(len(sections), 1))(*sections)
    return arr, ctypes.addressof(arr)


def _axes_args(q, k, wq, wk, cos, sin, positions, sections):
    dev, tables, sizes, _, _, held = _qk_args(q, k, wq, wk, cos, sin, None)
    sections = tuple(int(n) for n in sections)
    axes, B, S = len(sections), sizes[0], sizes[1]
    if not 1 <= axes <= 4 or min(sections) < 0 or 2 * sum(sections) != sizes[5]:
        _bad("sections: expected 1 to 4 numbers of pairs that add up to the tables' columns")
    bits = _index(positions, "positions", dev)
    if positions.shape == (axes, B, S):
        axis_stride, stride = B * S, S
    elif positions.shape == (axes, S) or positions.shape == (axes, 1, S):
        axis_stride, stride = S, 0
    else:
        _bad("positions: expected [axes, B, S] or [axes, S]")
    sec = _sections(sections)
    return dev, (*tables[:4], positions.data_ptr()), sizes, (sec[1], axes, axis_stride, stride), bits, (held, sec)


def qk_norm_rope_axes_forward(q, k, wq, wk, cos, sin, positions, sections, eps: float = 1e-6,
                              interleaved: bool = False, status=None, stream=None):
    """qk_norm_rope_forward for positions with several axes (time, height and width of patches).

    positions: int [axes, B, S] or [axes, S], a position on each axis; sections: how many of the
    rotated pairs belong to each axis, in order (1 to 4 numbers that add up to R / 2); cos, sin:
    fp32 [P, R / 2], column i for pair i (rope_axes_table). All else as in qk_norm_rope_forward."""
    if stream is not None:
        with _using(stream, q):
            return qk_norm_rope_axes_forward(q, k, wq, wk, cos, sin, positions, sections, eps, interleaved, status)
    dev, tables, sizes, ax, bits, held = _axes_args(q, k, wq, wk, cos, sin, positions, sections)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return qk_norm_rope_axes_forward(q, k, wq, wk, cos, sin, positions, sections, eps, interleaved, status)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _raise(_core.load().dash_qk_norm_rope_axes_fwd(
        q.data_ptr(), k.data_ptr(), *tables, q_out.data_ptr(), k_out.data_ptr(), _status_word(status, dev),
        *sizes, *ax, eps, interleaved, _DTYPE[q.dtype], bits, _stream(dev)), "dash_qk_norm_rope_axes_fwd")
    return q_out, k_out


def qk_norm_rope_axes_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, sections, eps: float = 1e-6,
                               interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None,
                               check: bool = True):
    """Gradients of qk_norm_rope_axes_forward with respect to q, k, wq and wk, as
    qk_norm_rope_backward returns them and with its workspace (new_qk_norm_rope_workspace)."""
    if stream is not None:
        with _using(stream, q):
            return qk_norm_rope_axes_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, sections, eps,
                                              interleaved, dq, dk, workspace, check=check)
    dev, tables, sizes, ax, bits, held = _axes_args(q, k, wq, wk, cos, sin, positions, sections)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return qk_norm_rope_axes_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, sections, eps,
                                              interleaved, dq, dk, workspace, check=check)
    dq, dk, dwq, dwk, ptrs, outs, workspace = _qk_grads(dq_out, dk_out, q, k, wq, wk, sizes, dq, dk, workspace, dev)
    _raise(_core.load().dash_qk_norm_rope_axes_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), *tables, *ptrs, *sizes, outs[0][1],
        outs[1][1], *ax, eps, interleaved, _DTYPE[q.dtype], bits, _stream(dev)), "dash_qk_norm_rope_axes_bwd")
    _finish(workspace, check, "dash_qk_norm_rope_axes_bwd")
    return dq, dk, dwq, dwk


# ---- gradient norm and clipping -----------------------------------------------------------------

class GradClipPlan:
    """The tensors of grad_clip and their table on the device. Holds the tensors, so that the
    addresses in the table stay theirs; build a new plan when a gradient is replaced, and keep
    the plan as long as a graph that captured a call on it is replayed."""

    def __init__(self, grads, outs, table, norm):
        self.grads, self.outs, self.table, self.norm = grads, outs, table, norm
        self.device = table.get_device()
        self.stream = _stream(self.device)           # that its memory was allocated on


def grad_clip_plan(grads, out=None, stream=None) -> GradClipPlan:
    """Plan of clipping `grads` (contiguous bf16, fp16 or fp32 CUDA tensors of one device, which
    overlap one another nowhere) in place, or into the tensors `out` of the same shapes and
    types."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if not grads or len(outs) != len(grads):
        _bad("grads: expected tensors, as many as out")
    if stream is not None:
        with _using(stream, grads[0]):
            return grad_clip_plan(grads, None if out is None else outs)
    dev = _device(grads[0], "grads[0]")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return grad_clip_plan(grads, None if out is None else outs)
    arr = (_ClipTensor * len(grads))()
    spans = set()
    for i, (g, o) in enumerate(zip(grads, outs)):
        for t, name in ((g, "grads"), (o, "out")):
            _on(t, f"{name}[{i}]", dev)
            if t.dtype not in _DTYPE or not t.is_contiguous():
                _bad(f"{name}[{i}]: expected contiguous bfloat16, float16 or float32")
            if t.numel():
                spans.add((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i))
        if o.dtype != g.dtype or o.shape != g.shape:
            _bad(f"out[{i}]: expected the type and shape of grads[{i}]")
        arr[i] = _ClipTensor(g.data_ptr(), o.data_ptr(), g.numel(), _DTYPE[g.dtype])
    spans = sorted(spans)
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        _bad("grads and out: tensors overlap")
    lib = _core.load()
    nbytes = lib.dash_grad_clip_plan_size(arr, len(grads))
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_grad_clip_plan_size")
    table = torch.empty(nbytes, dtype=torch.uint8, device=grads[0].device)
    _raise(lib.dash_grad_clip_plan(arr, len(grads), table.data_ptr(), nbytes, _stream(dev)),
           "dash_grad_clip_plan")
    return GradClipPlan(grads, outs, table, torch.empty((), dtype=_F32, device=grads[0].device))


def grad_clip(plan: GradClipPlan, max_norm: float, stream=None):
    """Global L2 norm of the plan's gradients, which are scaled by max_norm / norm when it is
    above max_norm. Returns (norm, tensors): norm is a device fp32 scalar that the next call
    overwrites."""
    if stream is not None:
        with _using(stream, plan.table):
            return grad_clip(plan, max_norm)
    if plan.device != _current_device():
        with torch.cuda.device(plan.device):
            return grad_clip(plan, max_norm)
    at = _stream(plan.device)
    if at != plan.stream:                            # its memory stays until this call's work has ended
        here = torch.cuda.current_stream(plan.device)
        plan.table.record_stream(here)
        plan.norm.record_stream(here)
    _raise(_core.load().dash_grad_clip(plan.table.data_ptr(), plan.table.nbytes, max_norm, plan.norm.data_ptr(),
                                       at), "dash_grad_clip")
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
    dev = _device(x, "x")
    if x.dtype != _BF16 or w.dtype != _BF16 or w.get_device() != dev:
        _bad(f"x and w: expected bfloat16 on cuda:{dev}")
    T, D, ldx = _rows(x, "x")
    V, Dw, ldw = _rows(w, "w")
    if Dw != D:
        _bad("w: expected as many columns as x")
    bits = _index(targets, "targets", dev)
    if targets.dim() != 1 or targets.numel() != T:
        _bad("targets: expected one index a row of x")
    return dev, bits, (T, V, D, ldx, ldw)


def linear_xent_forward(x, w, targets, ignore_index: int = -100, scale: float = 1.0, workspace=None,
                        stream=None, check: bool = True):
    """Softmax cross entropy of the logits scale * x w^T, which are never stored.

    x: bf16 [T, D] hidden states, w: bf16 [V, D] output embedding, targets: int [T].
    Returns (loss, lse), fp32 [T]; rows whose target is ignore_index have loss 0."""
    if stream is not None:
        with _using(stream, x):
            return linear_xent_forward(x, w, targets, ignore_index, scale, workspace, check=check)
    dev, bits, sizes = _xent_args(x, w, targets)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return linear_xent_forward(x, w, targets, ignore_index, scale, workspace, check=check)
    T = sizes[0]
    if workspace is None:
        workspace = new_linear_xent_workspace(*sizes[:3], x.device)
    loss = torch.empty(T, dtype=_F32, device=x.device)
    lse = loss.new_empty(T)
    ws, nbytes = _ws(workspace, dev)
    _raise(_core.load().dash_linear_xent_fwd(
        x.data_ptr(), w.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(), ws, nbytes, *sizes,
        scale, ignore_index, bits, _stream(dev)), "dash_linear_xent_fwd")
    _finish(workspace, check, "dash_linear_xent_fwd")
    return loss, lse


def linear_xent_backward(x, w, targets, lse, dloss, ignore_index: int = -100, scale: float = 1.0,
                         dw=None, accumulate: bool = False, dw_dtype=None, workspace=None, stream=None,
                         check: bool = True):
    """Gradients of sum(dloss * loss) with respect to x (bf16 [T, D]) and w.

    lse: from linear_xent_forward; dloss: fp32 [T]. dw: an optional [V, D] bf16 or fp32
    tensor to write to, or to add to with accumulate=True (tied embeddings, several
    micro-batches); else one of dw_dtype (bf16) is allocated. Returns (dx, dw)."""
    if stream is not None:
        with _using(stream, x):
            return linear_xent_backward(x, w, targets, lse, dloss, ignore_index, scale, dw, accumulate, dw_dtype,
                                        workspace, check=check)
    dev, bits, sizes = _xent_args(x, w, targets)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return linear_xent_backward(x, w, targets, lse, dloss, ignore_index, scale, dw, accumulate, dw_dtype,
                                        workspace, check=check)
    T, V, D = sizes[:3]
    plse, pdloss = _vector(lse, "lse", T, dev), _vector(dloss, "dloss", T, dev)
    if dw is None:
        if accumulate:
            _bad("accumulate: needs dw")
        dw = torch.empty((V, D), dtype=dw_dtype or _BF16, device=x.device)
    if dw.dtype not in (_BF16, _F32) or dw.shape != (V, D) or not dw.is_contiguous() or dw.get_device() != dev:
        _bad(f"dw: expected contiguous bfloat16 or float32 [V, D] on cuda:{dev}")
    if workspace is None:
        workspace = new_linear_xent_workspace(T, V, D, x.device)
    dx = x.new_empty((T, D))
    ws, nbytes = _ws(workspace, dev)
    _raise(_core.load().dash_linear_xent_bwd(
        x.data_ptr(), w.data_ptr(), targets.data_ptr(), plse, pdloss, dx.data_ptr(), dw.data_ptr(), ws, nbytes,
        *sizes, scale, ignore_index, bits, _DTYPE[dw.dtype], accumulate, _stream(dev)),
        "dash_linear_xent_bwd")
    _finish(workspace, check, "dash_linear_xent_bwd")
    return dx, dw


# ---- cross attention ----------------------------------------------------------------------------

def dash_cross_attn_fwd_workspace_size(B: int, Sq: int, Sk: int, Hq: int, Hk: int, D: int) -> int:
    return int(_core.load().dash_cross_attn_fwd_workspace_size(B, Sq, Sk, Hq, Hk, D))


def dash_cross_attn_bwd_workspace_size(B: int, Sq: int, Sk: int, Hq: int, Hk: int, D: int) -> int:
    return int(_core.load().dash_cross_attn_bwd_workspace_size(B, Sq, Sk, Hq, Hk, D))


def new_cross_attn_workspace(B: int, Sq: int, Sk: int, Hq: int, Hk: int, D: int, device,
                             forward_only: bool = False) -> torch.Tensor:
    """A workspace of cross_attn_forward and, unless forward_only, of cross_attn_backward (uint8)."""
    B = max(B, 1)                                    # (the sizes are those of at least one batch)
    nbytes = dash_cross_attn_fwd_workspace_size(B, Sq, Sk, Hq, Hk, D)
    if nbytes and not forward_only:
        nbytes = max(nbytes, dash_cross_attn_bwd_workspace_size(B, Sq, Sk, Hq, Hk, D))
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_cross_attn_fwd_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _cross_args(q, k, v, kv_lens):
    dev = _device(q, "q")
    if q.dtype != _BF16:
        _bad("q: expected bfloat16")
    B, Sq, Hq, D, qs = _heads(q, "q", _BF16, dev)
    Bk, Sk, Hk, Dk, ks = _heads(k, "k", _BF16, dev)
    Bv, Sv, Hv, Dv, vs = _heads(v, "v", _BF16, dev)
    if Bk != B or Dk != D or Hk < 1 or Hq % Hk:
        _bad("k: expected [B, Sk, Hk, D] with the B and D of q and a divisor of its heads")
    if (Bv, Sv, Hv, Dv) != (Bk, Sk, Hk, Dk):
        _bad("v: expected the shape of k")
    lens, bits = None, 32
    if kv_lens is not None:
        bits = _index(kv_lens, "kv_lens", dev)
        if kv_lens.dim() != 1 or kv_lens.numel() != B:
            _bad("kv_lens: expected one length a batch")
        lens = kv_lens.data_ptr()
    return dev, lens, bits, (B, Sq, Sk, Hq, Hk, D), (qs, ks, vs)


def cross_attn_forward(q, k, v, scale: float, kv_lens=None, workspace=None, status=None, stream=None):
    """Attention of queries to the keys and values of states of another length.

    q: bf16 [B, Sq, Hq, D]; k, v: bf16 [B, Sk, Hk, D], Hk a divisor of Hq, D contiguous, any strides
    that are multiples of 8 (parts of a fused projection, transposed [B, H, S, D], expanded batches
    or heads). kv_lens: int [B], how many of the Sk keys each batch has (None: all; 0: its rows are
    O = 0, LSE = -inf); what lies behind them is never used. status as in embed_forward: it reads
    DASH_ERR_BOUNDS when a length was out of range (its rows are NaN). Returns (o, lse): contiguous
    bf16 [B, Sq, Hq, D] and fp32 [B, Hq, Sq]."""
    if stream is not None:
        with _using(stream, q):
            return cross_attn_forward(q, k, v, scale, kv_lens, workspace, status)
    dev, lens, bits, sizes, held = _cross_args(q, k, v, kv_lens)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return cross_attn_forward(q, k, v, scale, kv_lens, workspace, status)
    o = torch.empty(q.shape, dtype=_BF16, device=q.device)
    lse = torch.empty((sizes[0], sizes[3], sizes[1]), dtype=_F32, device=q.device)
    if workspace is None and o.numel():
        workspace = new_cross_attn_workspace(*sizes, q.device, forward_only=True)
    ws, nbytes = (None, 0) if workspace is None else _ws(workspace, dev)
    _raise(_core.load().dash_cross_attn_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), lens, o.data_ptr(), lse.data_ptr(), _status_word(status, dev), ws,
        nbytes, *sizes, held[0][1], held[1][1], held[2][1], scale, bits, _stream(dev)), "dash_cross_attn_fwd")
    return o, lse


def cross_attn_backward(q, k, v, o, do, lse, scale: float, kv_lens=None, dq=None, dk=None, dv=None, workspace=None,
                        stream=None, check: bool = True):
    """Gradients of cross_attn_forward with respect to q, k and v.

    o and lse as the forward returned them, do contiguous like o. dq, dk, dv: optional tensors to
    write to, strided like q, k and v may be (parts of a fused projection's gradient), without
    strides of zero, and apart from all that the call reads and from one another. Rows of dk and dv behind a length are zero. Returns (dq, dk, dv)."""
    if stream is not None:
        with _using(stream, q):
            return cross_attn_backward(q, k, v, o, do, lse, scale, kv_lens, dq, dk, dv, workspace, check=check)
    dev, lens, bits, sizes, held = _cross_args(q, k, v, kv_lens)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return cross_attn_backward(q, k, v, o, do, lse, scale, kv_lens, dq, dk, dv, workspace, check=check)
    for t, name in ((o, "o"), (do, "do")):
        if t.dtype != _BF16 or t.shape != q.shape or not t.is_contiguous() or t.get_device() != dev:
            _bad(f"{name}: expected contiguous bfloat16 of the shape of q on cuda:{dev}")
    if (lse.dtype != _F32 or lse.shape != (sizes[0], sizes[3], sizes[1]) or not lse.is_contiguous()
            or lse.get_device() != dev):
        _bad(f"lse: expected contiguous float32 [B, Hq, Sq] on cuda:{dev}")
    taken = None
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        if t is not None and t.numel() and 0 not in t.stride():      # (those are refused below)
            taken = taken or {x.data_ptr() for x in (q, k, v, o, do)}
            if t.data_ptr() in taken:
                _bad(f"{name}: lies over another tensor of the call")
            taken.add(t.data_ptr())
    dq = torch.empty(q.shape, dtype=_BF16, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=_BF16, device=q.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=_BF16, device=q.device) if dv is None else dv
    outs = [_heads(t, n, _BF16, dev) for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"))]
    if outs[0][:4] != q.shape or outs[1][:4] != k.shape or outs[2][:4] != v.shape:
        _bad("dq, dk and dv: expected the shapes of q, k and v")
    if workspace is None:
        if not q.numel() and not k.numel():
            return dq, dk, dv
        nbytes = dash_cross_attn_bwd_workspace_size(*sizes)
        if nbytes == 0:
            raise DashError(DASH_ERR_UNSUPPORTED, "dash_cross_attn_bwd_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    ws, nbytes = _ws(workspace, dev)
    _raise(_core.load().dash_cross_attn_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), lens, o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), ws, nbytes, *sizes, held[0][1], held[1][1], held[2][1], outs[0][4][1],
        outs[1][4][1], outs[2][4][1], scale, bits, _stream(dev)), "dash_cross_attn_bwd")
    _finish(workspace, check, "dash_cross_attn_bwd")
    return dq, dk, dv


# ---- group norm with an activation --------------------------------------------------------------

def dash_group_norm_workspace_size(N: int, S: int, C: int, groups: int) -> int:
    return int(_core.load().dash_group_norm_workspace_size(int(N), int(S), int(C), int(groups)))


def new_group_norm_workspace(N: int, S: int, C: int, groups: int, device) -> torch.Tensor:
    """The workspace of group_norm_act_forward and _backward for N samples of S rows (uint8)."""
    nbytes = dash_group_norm_workspace_size(N, S, C, groups)
    if nbytes == 0:
        raise DashError(DASH_ERR_UNSUPPORTED, "dash_group_norm_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=1024)
def _row_strides(sample: int, row: int):
    arr = _c2(sample, row)
    return arr, ctypes.addressof(arr)


def _gn_args(x, w, b, groups, activation):
    dev = _device(x, "x")
    dtype, act = _DTYPE.get(x.dtype), _ACT.get(activation)
    if dtype is None:
        _bad("x: expected bfloat16, float16 or float32")
    if act is None:
        _bad("activation: expected 'none' or 'silu'")
    if x.dim() < 2:
        _bad("x: expected [N, ..., C]")
    shape, st = x.shape, x.stride()
    N, C = shape[0], shape[-1]
    if C < 1 or groups < 1 or C % groups:
        _bad("groups: expected a divisor of the channels")
    if st[-1] != 1 and C > 1:
        _bad("x: expected contiguous channels")
    # the dimensions between are one dimension of rows, the same number of elements apart
    S, row = 1, 0
    for n, step in zip(reversed(shape[1:-1]), reversed(st[1:-1])):
        if n == 1:
            continue
        if S > 1 and step != row * S:
            _bad("x: expected rows evenly spaced over the dimensions between N and C")
        if S == 1:
            row = step
        S *= n
    pw = None if w is None else _vector(w, "w", C, dev)
    pb = None if b is None else _vector(b, "b", C, dev)
    return dev, pw, pb, (N, S, C, groups), _row_strides(st[0] if N > 1 else 0, row), act, dtype


def _in_place_or_apart(out, name, t, other):
    """An output may lie over an input element for element, not otherwise."""
    if out.data_ptr() == t.data_ptr() and t.is_contiguous() or not t.numel():
        return
    end = t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    if out.data_ptr() < end and t.data_ptr() < out.data_ptr() + out.element_size() * out.numel():
        _bad(f"{name}: overlaps {other} other than element for element")


def group_norm_act_forward(x, w, b, groups: int, eps: float = 1e-5, activation="silu", out=None, workspace=None,
                           stream=None):
    """Group norm over channels-last x with the activation behind it: act(xh * w + b).

    x: [N, ..., C] bf16, fp16 or fp32 with contiguous channels; the dimensions between (rows, or
    height and width) are normed over together with the C / groups channels of a group, and may be
    strided as one (a part of a buffer with more channels). w, b: fp32 [C] or None; activation:
    "silu" or "none". out: an optional contiguous tensor to write to, which may be x itself. Returns
    (y, mean, rstd): contiguous y of x's type, fp32 [N, groups]."""
    if stream is not None:
        with _using(stream, x):
            return group_norm_act_forward(x, w, b, groups, eps, activation, out, workspace)
    dev, pw, pb, sizes, xs, act, dtype = _gn_args(x, w, b, groups, activation)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return group_norm_act_forward(x, w, b, groups, eps, activation, out, workspace)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.dtype != x.dtype or out.shape != x.shape or not out.is_contiguous() or out.get_device() != dev:
        _bad(f"out: expected contiguous, of the type and shape of x, on cuda:{dev}")
    else:
        _in_place_or_apart(out, "out", x, "x")
    mean = torch.empty((sizes[0], groups), dtype=_F32, device=x.device)
    rstd = torch.empty((sizes[0], groups), dtype=_F32, device=x.device)
    if workspace is None:
        workspace = new_group_norm_workspace(*sizes, x.device)
    _raise(_core.load().dash_group_norm_fwd(
        x.data_ptr(), pw, pb, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), *_ws(workspace, dev), *sizes, xs[1],
        eps, act, dtype, _stream(dev)), "dash_group_norm_fwd")
    return out, mean, rstd


def group_norm_act_backward(dy, x, w, b, mean, rstd, groups: int, activation="silu", dx=None, workspace=None,
                            stream=None):
    """Gradients of group_norm_act_forward with respect to x, w and b.

    dy: contiguous, of x's type and shape; mean, rstd: as the forward returned them. dx: an optional
    contiguous tensor to write to, which may be dy or a contiguous x itself. Returns (dx, dw, db), the
    last two fp32 [C] (None where w or b is None)."""
    if stream is not None:
        with _using(stream, x):
            return group_norm_act_backward(dy, x, w, b, mean, rstd, groups, activation, dx, workspace)
    dev, pw, pb, sizes, xs, act, dtype = _gn_args(x, w, b, groups, activation)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return group_norm_act_backward(dy, x, w, b, mean, rstd, groups, activation, dx, workspace)
    given = dx is not None
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    for t, name in ((dy, "dy"), (dx, "dx")):
        if t.dtype != x.dtype or t.shape != x.shape or not t.is_contiguous() or t.get_device() != dev:
            _bad(f"{name}: expected contiguous, of the type and shape of x, on cuda:{dev}")
    if given:
        _in_place_or_apart(dx, "dx", x, "x")
        _in_place_or_apart(dx, "dx", dy, "dy")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != _F32 or t.shape != (sizes[0], groups) or not t.is_contiguous() or t.get_device() != dev:
            _bad(f"{name}: expected contiguous float32 [N, groups] on cuda:{dev}")
    dw = pdw = db = pdb = None
    if w is not None:
        dw = torch.empty(sizes[2], dtype=_F32, device=x.device)
        pdw = dw.data_ptr()
    if b is not None:
        db = torch.empty(sizes[2], dtype=_F32, device=x.device)
        pdb = db.data_ptr()
    if workspace is None:
        workspace = new_group_norm_workspace(*sizes, x.device)
    _raise(_core.load().dash_group_norm_bwd(
        dy.data_ptr(), x.data_ptr(), pw, pb, mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), pdw, pdb,
        *_ws(workspace, dev), *sizes, xs[1], act, dtype, _stream(dev)), "dash_group_norm_bwd")
    return dx, dw, db
