"""CPU: cross attention, the rotation over several axes and the group norm refuse bad arguments
before anything reaches the device, and run on their tensors' device whichever is current."""
import ctypes

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built
from tests.test_train_abi import INV, QK_BWD, QK_FWD, SMALL, UNS, _call
from tests.test_train_devices import library, on1  # noqa: F401


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    return da.load()


S3, S2, I3 = ctypes.c_longlong * 3, ctypes.c_longlong * 2, ctypes.c_int * 3


def _strides(H, D=64, S=40):
    return S3(S * H * D, H * D, D)


CROSS_FWD = dict(q=16, k=16, v=16, lens=16, o=16, lse=16, status=None, ws=256, wsb=1 << 30, B=2, Sq=4, Sk=4000, Hq=4,
                 Hk=2, D=64, qs=_strides(4, S=4), ks=_strides(2), vs=_strides(2), scale=0.1, bits=32, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(o=None), INV), (dict(lse=None), INV),
    (dict(B=-1), INV), (dict(Sq=-1), INV), (dict(Sk=-1), INV), (dict(Hq=0), INV), (dict(Hk=3), INV), (dict(Hk=0), INV),
    (dict(D=0), INV), (dict(D=60), UNS), (dict(D=136), UNS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(bits=16), INV), (dict(qs=None), INV),
    (dict(vs=None), INV), (dict(ks=S3(0, 60, 64)), UNS), (dict(qs=S3(-8, 64, 64)), UNS), (dict(ks=S3(0, 0, 64)), UNS),
    (dict(q=8), INV), (dict(k=24), INV), (dict(o=20), INV), (dict(lse=2), INV), (dict(lens=2), INV),
    (dict(lens=20, bits=64), INV), (dict(status=2), INV), (dict(ws=128), INV), (dict(ws=None), INV),
    (dict(wsb=100), SMALL), (dict(Sq=2 ** 25), UNS), (dict(B=2 ** 19, Hq=2 ** 12, Hk=2), UNS)])
def test_cross_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_cross_attn_fwd, CROSS_FWD, **kw) == want


CROSS_BWD = dict(q=16, k=16, v=16, lens=16, o=16, do=16, lse=16, dq=16, dk=16, dv=16, ws=256, wsb=1 << 30, B=2, Sq=4,
                 Sk=40, Hq=4, Hk=2, D=64, qs=_strides(4, S=4), ks=_strides(2), vs=_strides(2), dqs=_strides(4, S=4),
                 dks=_strides(2), dvs=_strides(2), scale=0.1, bits=32, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(do=None), INV), (dict(dq=None), INV), (dict(dk=None), INV), (dict(dv=None), INV), (dict(o=None), INV),
    (dict(ws=None), INV), (dict(ws=64), INV), (dict(wsb=100), SMALL), (dict(wsb=1024), SMALL), (dict(dqs=None), INV),
    (dict(dks=S3(0, 128, 64)), INV), (dict(dvs=S3(5120, 128, 0)), INV), (dict(dqs=S3(1024, 0, 64)), UNS),
    (dict(dks=S3(5120, 100, 64)), UNS), (dict(dq=8), INV), (dict(dv=4), INV), (dict(D=12), UNS), (dict(scale=0.0), INV)])
def test_cross_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_cross_attn_bwd, CROSS_BWD, **kw) == want


def test_cross_workspace_sizes(lib):
    # one key tile, many rows: nothing but the rows' numbers and, where rows are cut, partials
    B, Sq, Sk, H, D = 4, 4096, 77, 16, 64
    rows = B * H * Sq
    fwd, bwd = (f(B, Sq, Sk, H, H, D) for f in (da.dash_cross_attn_fwd_workspace_size,
                                               da.dash_cross_attn_bwd_workspace_size))
    assert fwd == 256
    assert 8 * rows <= bwd <= 256 + 8 * rows + 32 * B * H * 128 * 2 * D * 4 and bwd % 256 == 0
    # a single token against many keys: ranges of keys leave partials of one row tile a group
    fwd = da.dash_cross_attn_fwd_workspace_size(7, 1, 1500, 32, 8, 128)
    assert 56 * 128 * 129 * 4 < fwd < 12 * 56 * 128 * 129 * 4 + 1024
    for bad in ((2, 4, 40, 3, 2, 64), (2, 4, 40, 4, 2, 60), (0, 4, 40, 4, 2, 64), (2, 4, 2 ** 25, 4, 2, 64)):
        assert da.dash_cross_attn_fwd_workspace_size(*bad) == 0
        assert da.dash_cross_attn_bwd_workspace_size(*bad) == 0
    with pytest.raises(da.DashError):
        da.new_cross_attn_workspace(2, 4, 40, 4, 2, 60, "cpu")


def _axes(d):
    a = dict(d)
    a.update(pos=16)
    out = {}
    for n, v in a.items():
        if n == "ps":
            out.update(sections=I3(8, 12, 12), axes=3, axs=4)
        out[n] = v
    return out


AXES_FWD, AXES_BWD = _axes(QK_FWD), _axes(QK_BWD)


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), INV), (dict(sections=None), INV), (dict(axes=0), INV), (dict(axes=5), INV), (dict(axes=2), INV),
    (dict(sections=I3(8, 12, 13)), INV), (dict(sections=I3(40, -8, 0)), INV), (dict(axs=-1), INV), (dict(q=None), INV),
    (dict(P=2 ** 31), UNS), (dict(R=62), INV), (dict(D=60, R=60), UNS), (dict(qo=None), INV), (dict(status=2), INV)])
def test_axes_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_qk_norm_rope_axes_fwd, AXES_FWD, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), INV), (dict(sections=I3(8, 12, 13)), INV), (dict(ws=None), INV), (dict(wsb=300), SMALL),
    (dict(dqs=S3(0, 128, 0)), INV), (dict(dks=None), INV), (dict(dqo=None), INV), (dict(dq=8), INV)])
def test_axes_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_qk_norm_rope_axes_bwd, AXES_BWD, **kw) == want


GN_FWD = dict(x=16, w=16, b=16, y=16, mean=16, rstd=16, ws=256, wsb=1 << 30, N=2, S=40, C=64, G=8, xs=S2(2560, 64),
              eps=1e-5, act=1, dtype=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(y=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV), (dict(N=-1), INV),
    (dict(S=-1), INV), (dict(C=0), INV), (dict(G=0), INV), (dict(G=7), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(act=2), INV), (dict(dtype=3), INV), (dict(xs=None), INV), (dict(x=17), INV),
    (dict(dtype=2, y=18), INV), (dict(w=2), INV), (dict(b=6), INV), (dict(ws=None), INV), (dict(ws=128), INV),
    (dict(wsb=256), SMALL), (dict(xs=S2(-1, 64)), UNS), (dict(C=2 ** 19, G=2 ** 10), UNS), (dict(C=8192, G=1), UNS),
    (dict(N=2 ** 24), UNS), (dict(S=2 ** 31), UNS)])
def test_group_norm_fwd_refuses(lib, kw, want):
    assert _call(lib.dash_group_norm_fwd, GN_FWD, **kw) == want


GN_BWD = dict(dy=16, x=16, w=16, b=16, mean=16, rstd=16, dx=16, dw=16, db=16, ws=256, wsb=1 << 30, N=2, S=40, C=64, G=8,
              xs=S2(2560, 64), act=1, dtype=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INV), (dict(x=None), INV), (dict(dx=None), INV), (dict(mean=None), INV), (dict(dy=17), INV),
    (dict(dw=2), INV), (dict(db=6), INV), (dict(act=-1), INV), (dict(wsb=100), SMALL)])
def test_group_norm_bwd_refuses(lib, kw, want):
    assert _call(lib.dash_group_norm_bwd, GN_BWD, **kw) == want


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q:"):
        da.cross_attn_forward(x, x, x, 1.0)
    with pytest.raises(ValueError, match="q:"):
        da.qk_norm_rope_axes_forward(x, x, None, None, torch.zeros(4, 8), torch.zeros(4, 8),
                                     torch.zeros(1, 1, 4, dtype=torch.int64), (8,))
    with pytest.raises(ValueError, match="x:"):
        da.group_norm_act_forward(x, None, None, 2)


def _cross():
    bf = dict(dtype=torch.bfloat16)
    return on1(torch.zeros(1, 4, 2, 16, **bf)), on1(torch.zeros(1, 9, 1, 16, **bf)), on1(torch.zeros(1, 9, 1, 16, **bf))


def _qk():
    w, c = on1(torch.ones(16)), on1(torch.zeros(8, 8))
    q, k, _ = _cross()
    return q, k[:, :4], w, w, c, c, on1(torch.zeros(2, 1, 4, dtype=torch.int64)), (3, 5)


def _gn():
    return on1(torch.zeros(2, 5, 16)), on1(torch.ones(16)), on1(torch.ones(16))


CALLS = {
    "dash_cross_attn_fwd": lambda: da.cross_attn_forward(*_cross(), 1.0),
    "dash_cross_attn_bwd": lambda: da.cross_attn_backward(*_cross(), _cross()[0], _cross()[0],
                                                          on1(torch.zeros(1, 2, 4)), 1.0),
    "dash_qk_norm_rope_axes_fwd": lambda: da.qk_norm_rope_axes_forward(*_qk()),
    "dash_qk_norm_rope_axes_bwd": lambda: da.qk_norm_rope_axes_backward(*_qk()[:2], *_qk()),
    "dash_group_norm_fwd": lambda: da.group_norm_act_forward(*_gn(), 4),
    "dash_group_norm_bwd": lambda: da.group_norm_act_backward(_gn()[0], *_gn(), on1(torch.zeros(2, 4)),
                                                              on1(torch.zeros(2, 4)), 4),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_runs_on_the_tensors_device(library, name, current):  # noqa: F811
    library.state["current"] = current
    CALLS[name]()
    assert name in [n for n, _ in library.calls]
    assert all(dev == 1 for n, dev in library.calls if not n.endswith("_size")), library.calls
    assert library.state["current"] == current
