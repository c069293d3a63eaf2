"""GPU: norm and rotation of queries and keys by positions with several axes, and the gradients,
against the float64 definition. The arithmetic is that of the one-axis operator, and so are the
tolerances (see test_qk_norm_rope.py): (D + 32) 2^-24 of the terms' absolute values, the result's
rounding, and for dw one more step a row."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu
from tests.test_qk_norm_rope import TINY, TYPES, _swap

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(B, S, Hq, Hk, D, sections, t, P=40, seed=0, weights=True, own_ladders=False, ids=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(B, S, Hq + 2 * Hk, D, generator=g, device="cuda").to(t)
    x = {"q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hk], "sections": sections}
    for n in "qk":
        x["w" + n] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda") if weights else None
    x["cos"], x["sin"] = da.rope_axes_table(P, sections, 1000.0, own_ladders)
    x["pos"] = torch.randint(0, P, (len(sections), B, S), generator=g, device="cuda").to(ids)
    x["dq"] = torch.randn(B, S, Hq, D, generator=g, device="cuda").to(t)
    x["dk"] = torch.randn(B, S, Hk, D, generator=g, device="cuda").to(t)
    return x


def _check(x, il, eps, outs=None, grads=None):
    D, R = x["q"].shape[-1], 2 * sum(x["sections"])
    rel = (D + 32) * 2.0 ** -24
    for i, n in enumerate("qk"):
        a, w, d = x[n], x["w" + n], x["d" + n]
        u = torch.finfo(a.dtype).eps / 2
        r = 1 / torch.sqrt((a.double() ** 2).mean(-1, keepdim=True) + eps)
        wd = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
        at = (x["cos"], x["sin"], x["pos"], x["sections"], eps, il)
        if outs is not None:
            want = ref.norm_rope_axes(a, w, *at)
            y = a.double() * r * wd
            tol = rel * (y.abs() + _swap(y, R, il)) + u * want.abs() * (1 + rel) + TINY[a.dtype]
            err = (outs[i].double() - want).abs()
            assert outs[i].is_contiguous() and bool((err <= tol).all()), (n, float((err - tol).max()))
        if grads is not None:
            dx, dw = ref.norm_rope_axes_grad(d, a, w, *at)
            nn = a.double() * r
            da_ = d.double().abs() + _swap(d.double(), R, il)
            ua = da_ * wd.abs()
            mag = r * (ua + nn.abs() * (ua * nn.abs()).mean(-1, keepdim=True))
            tol = 2 * rel * mag + u * dx.abs() * (1 + rel) + TINY[a.dtype]
            err = (grads[i].double() - dx).abs()
            assert bool((err <= tol).all()), (n, float((err - tol).max()))
            if w is None:
                assert grads[2 + i] is None
            else:
                rows = a.shape[0] * a.shape[1] * a.shape[2]
                tol = (rows + D + 32) * 2.0 ** -24 * (da_ * nn.abs()).sum((0, 1, 2)) + 2.0 ** -149
                assert bool(((grads[2 + i].double() - dw).abs() <= tol).all()), n


def _both(x, il, eps=1e-6, **kw):
    a = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], x["sections"])
    outs = da.qk_norm_rope_axes_forward(x["q"], x["k"], *a, eps=eps, interleaved=il)
    grads = da.qk_norm_rope_axes_backward(x["dq"], x["dk"], x["q"], x["k"], *a, eps=eps, interleaved=il, **kw)
    return outs, grads


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hk,D,sections", [
    (1, 1, 1, 1, 8, (4,)), (2, 3, 4, 2, 64, (8, 12, 12)), (1, 33, 5, 1, 128, (16, 24, 24)),
    (2, 17, 3, 3, 96, (10, 20, 18)), (1, 20, 4, 2, 80, (3, 5, 8)), (1, 9, 2, 1, 256, (32, 32, 63, 1)),
    (2, 5, 7, 2, 128, (7, 3)), (1, 6, 3, 1, 96, (0, 12, 0, 0)), (1, 4, 2, 2, 64, (0, 1)), (3, 2, 2, 1, 128, (22, 21, 21)),
    (1, 5, 3, 2, 128, (0, 0))])
def test_matches_definition(t, il, B, S, Hq, Hk, D, sections):
    x = _inputs(B, S, Hq, Hk, D, sections, t, seed=D + S)
    outs, grads = _both(x, il)
    _check(x, il, 1e-6, outs, grads)


@pytest.mark.parametrize("il", [False, True])
def test_many_rows_own_ladders_and_int32(il):
    x = _inputs(2, 1500, 32, 8, 64, (6, 13, 13), torch.bfloat16, P=3000, seed=3, own_ladders=True, ids=torch.int32)
    outs, grads = _both(x, il)
    _check(x, il, 1e-6, outs, grads)


@pytest.mark.parametrize("il", [False, True])
def test_one_axis_gives_the_one_axis_operators_bits(il):
    """With one axis, or the same position on every axis, the results are those of qk_norm_rope."""
    x = _inputs(2, 40, 6, 2, 128, (64,), torch.bfloat16, seed=5)
    outs, grads = _both(x, il)
    one = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"][0])
    want = da.qk_norm_rope_forward(x["q"], x["k"], *one, interleaved=il)
    gwant = da.qk_norm_rope_backward(x["dq"], x["dk"], x["q"], x["k"], *one, interleaved=il)
    y = dict(x, sections=(5, 20, 39), pos=x["pos"].expand(3, 2, 40).contiguous())
    outs3, grads3 = _both(y, il)
    for a, b, c in zip(outs + grads, want + gwant, outs3 + grads3):
        assert torch.equal(a, b) and torch.equal(c, b)


def test_position_out_of_range_on_one_axis():
    x = _inputs(1, 12, 2, 1, 64, (8, 12, 12), torch.bfloat16, P=30, seed=7)
    want, gwant = _both(x, False)
    x["pos"] = x["pos"].clone()
    x["pos"][2, 0, 5] = 30
    x["pos"][0, 0, 6] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"], x["sections"])
    outs = da.qk_norm_rope_axes_forward(x["q"], x["k"], *a, status=status)
    assert int(status) == da.DASH_ERR_BOUNDS
    ws = da.new_qk_norm_rope_workspace(1, 12, 2, 1, 64, "cuda")
    grads = da.qk_norm_rope_axes_backward(x["dq"], x["dk"], x["q"], x["k"], *a, workspace=ws, check=False)
    assert da.dash_attn_get_status(ws) == da.DASH_ERR_BOUNDS and "a position" in da.dash_last_error()
    keep = [0, 1, 2, 3, 4, 7, 8, 9, 10, 11]
    for got, w in zip(outs + grads[:2], want + gwant[:2]):
        assert bool(torch.isnan(got[:, 5:7]).all()) and torch.equal(got[:, keep], w[:, keep])


def test_strides_positions_by_row_and_gradients_in_place():
    x = _inputs(2, 19, 4, 2, 128, (16, 24, 24), torch.bfloat16, seed=5)
    x["pos"] = x["pos"][:, :1].expand(3, 2, 19).contiguous()
    want, gwant = _both(x, False)
    for pos in (x["pos"][:, 0].contiguous(), x["pos"][:, :1].contiguous()):
        got, _ = _both(dict(x, pos=pos), False)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    y = dict(x, q=x["q"].transpose(1, 2).contiguous().transpose(1, 2))
    fused = torch.full((2, 19, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got, ggot = _both(y, False, dq=fused[:, :, :4], dk=fused[:, :, 4:6])
    assert all(torch.equal(a, b) for a, b in zip(want + gwant, got + ggot)) and bool((fused[:, :, 6:] == 7).all())


def test_empty_reproducible_and_graph():
    x = _inputs(2, 700, 16, 4, 128, (9, 12, 11), torch.bfloat16, seed=8)
    e = {n: x[n][:, :0] for n in ("q", "k", "dq", "dk")}
    outs, grads = _both(dict(x, **e, pos=x["pos"][:, :, :0].contiguous()), False)
    assert outs[0].shape == (2, 0, 16, 128) and not bool(grads[2].any())
    ws = da.new_qk_norm_rope_workspace(2, 700, 16, 4, 128, "cuda")
    outs, grads = _both(x, True, workspace=ws)
    want = outs + grads
    for _ in range(3):
        ws.random_(0, 255)
        outs, grads = _both(x, True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, outs + grads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs, grads = _both(x, True, workspace=ws, check=False)
    for t in outs + grads:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs + grads))


def test_refusals():
    x = _inputs(1, 4, 2, 1, 64, (8, 12, 12), torch.bfloat16)
    a = (x["q"], x["k"], x["wq"], x["wk"], x["cos"], x["sin"])
    for sections in ((8, 12, 11), (8, 12, 13), (40, -8), (8, 8, 8, 4, 4), ()):
        with pytest.raises(ValueError, match="sections"):
            da.qk_norm_rope_axes_forward(*a, x["pos"], sections)
    for pos in (x["pos"][:2], x["pos"][:, :, :3], x["pos"].float(), x["pos"][:, 0, 0]):
        with pytest.raises(ValueError, match="positions"):
            da.qk_norm_rope_axes_forward(*a, pos, x["sections"])
