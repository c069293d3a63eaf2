"""CPU: the training-step operators refuse bad arguments before anything reaches the device."""
import ctypes

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built

INV, UNS, SMALL = da.DASH_ERR_INVALID_ARG, da.DASH_ERR_UNSUPPORTED, da.DASH_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    return da.load()


def _call(f, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    return f(*a.values())


EMBED_FWD = dict(table=16, ids=16, out=16, status=None, T=4, V=10, D=8, ldt=8, ldo=8, scale=1.0, dtype=0,
                 bits=64, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), INV), (dict(ids=None), INV), (dict(out=None), INV), (dict(T=-1), INV), (dict(V=0), INV),
    (dict(D=0), INV), (dict(ldt=7), INV), (dict(ldo=7), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV),
    (dict(bits=16), INV), (dict(table=17), INV), (dict(ids=20), INV), (dict(dtype=2, out=18), INV),
    (dict(status=18), INV), (dict(T=2 ** 31), UNS), (dict(V=2 ** 31), UNS), (dict(D=2 ** 21, ldt=2 ** 21, ldo=2 ** 21), UNS)])
def test_embed_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_embed_fwd, EMBED_FWD, **kw) == want


EMBED_BWD = dict(dout=16, ids=16, dtable=16, ws=256, wsb=1 << 30, T=4, V=10, D=8, ld=8, scale=1.0, pad=-1, acc=0,
                 dt=0, tt=0, bits=64, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dout=None), INV), (dict(ids=None), INV), (dict(dtable=None), INV), (dict(ws=None), INV),
    (dict(ws=128), INV), (dict(T=-1), INV), (dict(ld=7), INV), (dict(pad=-2), INV), (dict(acc=2), INV),
    (dict(dt=3), INV), (dict(tt=7), INV), (dict(dt=0, tt=1), UNS), (dict(dt=2, tt=0), UNS), (dict(bits=8), INV),
    (dict(wsb=256), SMALL), (dict(T=2 ** 31), UNS)])
def test_embed_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_embed_bwd, EMBED_BWD, **kw) == want


def test_workspace_sizes(lib):
    T, V, D = 1000, 5000, 72
    need = 256 + 4 * T * 4 + 2 * 32 * D * 4
    assert need <= da.dash_embed_bwd_workspace_size(T, V, D) <= need + 8 * 256
    assert da.dash_embed_bwd_workspace_size(-1, 5, 8) == 0 and da.dash_embed_bwd_workspace_size(1, 0, 8) == 0
    assert da.dash_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 264) == 0
    assert da.dash_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 128) > 0
    assert da.dash_linear_xent_workspace_size(10, 10, 12) == 0
    assert da.dash_linear_xent_workspace_size(10, 10, 16) > 0
    # the logits' gradient never takes more than a piece, however large the vocabulary
    assert da.dash_linear_xent_workspace_size(8192, 1 << 20, 64) < 1 << 30


S3 = (ctypes.c_longlong * 3)
QK_FWD = dict(q=16, k=16, wq=16, wk=16, cos=16, sin=16, pos=16, qo=16, ko=16, status=None, B=1, S=4, Hq=2, Hk=1,
              D=64, R=64, P=8, qs=S3(0, 128, 64), ks=S3(0, 64, 64), ps=4, eps=1e-6, il=0, dtype=0, bits=64,
              stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(cos=None), INV), (dict(qo=None), INV), (dict(ko=None), INV),
    (dict(B=-1), INV), (dict(R=63), INV), (dict(R=66), INV), (dict(R=-2), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(il=2), INV), (dict(dtype=5), INV), (dict(bits=1), INV), (dict(D=0, R=0), INV),
    (dict(D=60, R=60), UNS), (dict(D=264, R=64), UNS), (dict(qs=S3(0, 130, 64)), UNS), (dict(ks=S3(0, -64, 64)), UNS),
    (dict(qs=None), INV), (dict(ps=-1), INV), (dict(q=24), INV), (dict(pos=20), INV), (dict(status=2), INV),
    (dict(B=2 ** 16, S=2 ** 15), UNS), (dict(P=-1), INV)])
def test_qk_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_qk_norm_rope_fwd, QK_FWD, **kw) == want


QK_BWD = dict(dqo=16, dko=16, q=16, k=16, wq=16, wk=16, cos=16, sin=16, pos=16, dq=16, dk=16, dwq=16, dwk=16,
              ws=256, wsb=1 << 30, B=1, S=4, Hq=2, Hk=1, D=64, R=64, P=8, qs=S3(0, 128, 64), ks=S3(0, 64, 64),
              dqs=S3(0, 128, 64), dks=S3(0, 64, 64), ps=4, eps=1e-6, il=0, dtype=0, bits=64, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dqo=None), INV), (dict(dk=None), INV), (dict(ws=None), INV), (dict(ws=64), INV), (dict(wsb=300), SMALL),
    (dict(dqs=None), INV), (dict(dks=S3(0, 60, 64)), UNS), (dict(dqs=S3(0, 128, 0)), INV), (dict(dks=S3(0, 0, 64)), INV), (dict(dwq=2), INV), (dict(dq=8), INV), (dict(R=1), INV)])
def test_qk_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_qk_norm_rope_bwd, QK_BWD, **kw) == want


XENT_FWD = dict(x=16, w=16, y=16, loss=16, lse=16, ws=256, wsb=1 << 40, T=4, V=10, D=64, ldx=64, ldw=64, scale=1.0,
                ign=-100, bits=64, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(loss=None), INV), (dict(lse=None), INV),
    (dict(ws=None), INV), (dict(ws=128), INV), (dict(wsb=100), SMALL), (dict(T=-1), INV), (dict(V=0), INV),
    (dict(D=0), INV), (dict(D=60, ldx=64), UNS), (dict(ldx=56), INV), (dict(ldw=68), UNS), (dict(scale=0.0), INV),
    (dict(scale=float("nan")), INV), (dict(bits=0), INV), (dict(x=24), INV), (dict(y=20), INV), (dict(T=2 ** 31), UNS)])
def test_xent_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_linear_xent_fwd, XENT_FWD, **kw) == want


XENT_BWD = dict(x=16, w=16, y=16, lse=16, dloss=16, dx=16, dw=16, ws=256, wsb=1 << 40, T=4, V=10, D=64, ldx=64,
                ldw=64, scale=1.0, ign=-100, bits=64, dwt=0, acc=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dx=None), INV), (dict(dw=None), INV), (dict(lse=None), INV), (dict(dloss=None), INV), (dict(dwt=1), INV),
    (dict(acc=-1), INV), (dict(dx=8), INV), (dict(dw=4), INV), (dict(wsb=100), SMALL), (dict(D=12, ldx=16), UNS)])
def test_xent_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_linear_xent_bwd, XENT_BWD, **kw) == want


def test_clip_refuses(lib):
    from reproducible_deterministic_attn_gb300.train_ops import _ClipTensor

    def plan(grad=16, out=16, n=8, dtype=0, count=1, where=256, size=1 << 20):
        t = (_ClipTensor * 1)(_ClipTensor(grad, out, n, dtype))
        return lib.dash_grad_clip_plan(t, count, where, size, None)

    assert lib.dash_grad_clip_plan(None, 1, 256, 1 << 20, None) == INV
    assert plan(count=0) == INV and plan(n=-1) == INV and plan(dtype=3) == INV and plan(grad=None) == INV
    assert plan(grad=17) == INV and plan(dtype=2, out=18) == INV and plan(where=128) == INV and plan(where=None) == INV
    assert plan(size=100) == SMALL and plan(n=2 ** 50) == UNS
    assert lib.dash_grad_clip_plan_size((_ClipTensor * 1)(_ClipTensor(16, 16, -1, 0)), 1) == 0
    clip = lambda plan=256, size=1 << 20, limit=1.0, norm=16: lib.dash_grad_clip(plan, size, limit, norm, None)
    assert clip(plan=None) == INV and clip(norm=None) == INV and clip(plan=128) == INV and clip(norm=2) == INV
    assert clip(limit=-1.0) == INV and clip(limit=float("nan")) == INV and clip(size=256) == SMALL


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="table"):
        da.embed_forward(x, i)
    with pytest.raises(ValueError, match="dout"):
        da.embed_backward(x, i, 4)
    with pytest.raises(ValueError, match="q:"):
        da.qk_norm_rope_forward(x[None, None], x[None, None], None, None, x, x)
    with pytest.raises(ValueError, match="x:"):
        da.linear_xent_forward(x, x, i)
    with pytest.raises(ValueError, match="grads"):
        da.grad_clip_plan([x])
    with pytest.raises(ValueError, match="expected tensors"):
        da.grad_clip_plan([])
