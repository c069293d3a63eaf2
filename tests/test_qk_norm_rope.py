"""GPU: norm and rotation of queries and keys, and the gradients, against the float64
definition.

Tolerances. Forward: the sum of D squares (D 2^-24), rsqrtf (2^-22), five products and a sum
in fp32 of |a c| + |b s|: (D + 32) 2^-24 relative to m = |y_a c| + |y_b s| with m <= |y_a| +
|y_b|, then the result's rounding u = eps / 2. Backward: dx = r (u - n mean(u n)): the same
relative error of r (|u| + |n| mean|u n|), each with its rotation; dw: `rows` terms in fp32 in
any grouping, (rows + D + 32) 2^-24 of the sum of absolute values."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

TYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(B, S, Hq, Hk, D, R, t, P=None, seed=0, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    P = P or S + 9
    qkv = torch.randn(B, S, Hq + 2 * Hk, D, generator=g, device="cuda").to(t)
    x = {"q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hk]}
    for n in "qk":
        x["w" + n] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda") if weights else None
    x["cos"], x["sin"] = da.rope_table(P, R, 1000.0)
    x["pos"] = torch.randint(0, P, (B, S), generator=g, device="cuda")
    x["dq"] = torch.randn(B, S, Hq, D, generator=g, device="cuda").to(t)
    x["dk"] = torch.randn(B, S, Hk, D, generator=g, device="cuda").to(t)
    return x


def _swap(a, R, il):
    """|.| of each column's rotation partner."""
    a = a.abs().clone()
    if R == 0:
        return torch.zeros_like(a)
    if il:
        p = torch.stack((a[..., 1:R:2], a[..., 0:R:2]), -1).flatten(-2)
    else:
        p = torch.cat((a[..., R // 2:R], a[..., :R // 2]), -1)
    return torch.cat((p, torch.zeros_like(a[..., R:])), -1)


def _check(x, R, il, eps, outs=None, grads=None, pos=None):
    pos = x["pos"].long() if pos is None else pos
    D = x["q"].shape[-1]
    rel = (D + 32) * 2.0 ** -24
    for i, n in enumerate("qk"):
        a, w, d = x[n], x["w" + n], x["d" + n]
        t = a.dtype
        u = torch.finfo(t).eps / 2
        r = 1 / torch.sqrt((a.double() ** 2).mean(-1, keepdim=True) + eps)
        wd = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
        if outs is not None:
            want = ref.norm_rope(a, w, x["cos"], x["sin"], pos, eps, il)
            y = a.double() * r * wd
            tol = rel * (y.abs() + _swap(y, R, il)) + u * want.abs() * (1 + rel) + TINY[t]
            err = (outs[i].double() - want).abs()
            assert outs[i].is_contiguous() and bool((err <= tol).all()), (n, float((err - tol).max()))
        if grads is not None:
            dx, dw = ref.norm_rope_grad(d, a, w, x["cos"], x["sin"], pos, eps, il)
            nn = a.double() * r
            da_ = d.double().abs() + _swap(d.double(), R, il)
            ua = da_ * wd.abs()
            mag = r * (ua + nn.abs() * (ua * nn.abs()).mean(-1, keepdim=True))
            tol = 2 * rel * mag + u * dx.abs() * (1 + rel) + TINY[t]
            err = (grads[i].double() - dx).abs()
            assert bool((err <= tol).all()), (n, float((err - tol).max()))
            rows = a.shape[0] * a.shape[1] * a.shape[2]
            if w is None:
                assert grads[2 + i] is None
            else:
                tol = (rows + D + 32) * 2.0 ** -24 * (da_ * nn.abs()).sum((0, 1, 2)) + 2.0 ** -149
                assert bool(((grads[2 + i].double() - dw).abs() <= tol).all()), n


def _both(x, il, eps=1e-6, **kw):
    a = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"])
    outs = da.qk_norm_rope_forward(x["q"], x["k"], *a, eps=eps, interleaved=il)
    grads = da.qk_norm_rope_backward(x["dq"], x["dk"], x["q"], x["k"], *a, eps=eps, interleaved=il, **kw)
    return outs, grads


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hk,D,R", [(1, 1, 1, 1, 8, 8), (2, 3, 4, 2, 64, 64), (1, 33, 5, 1, 128, 128),
                                           (2, 17, 3, 3, 96, 96), (1, 20, 4, 2, 80, 32), (1, 9, 2, 1, 256, 256),
                                           (2, 5, 7, 2, 128, 20), (1, 6, 3, 1, 96, 24), (1, 4, 2, 2, 64, 2),
                                           (3, 2, 2, 1, 200, 100), (1, 5, 3, 2, 128, 0)])
def test_matches_definition(t, il, B, S, Hq, Hk, D, R):
    x = _inputs(B, S, Hq, Hk, D, R, t, seed=D + R + S)
    outs, grads = _both(x, il)
    _check(x, R, il, 1e-6, outs, grads)


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("t", TYPES)
def test_many_rows(t, il):
    """Enough rows that a warp has several heads in flight and blocks walk over several items."""
    x = _inputs(2, 1500, 32, 8, 64, 64, t, seed=3)
    outs, grads = _both(x, il)
    _check(x, 64, il, 1e-6, outs, grads)


def test_no_weights_positions_by_row_and_default():
    x = _inputs(3, 11, 4, 2, 64, 64, torch.bfloat16, seed=4, weights=False)
    outs, grads = _both(x, False)
    _check(x, 64, False, 1e-6, outs, grads)
    base = torch.arange(11, device="cuda")
    for given, used in ((None, base), (base.int() + 5, base + 5), (base[None] + 2, base + 2)):
        outs = da.qk_norm_rope_forward(x["q"], x["k"], None, None, x["cos"], x["sin"], given)
        _check(x, 64, False, 1e-6, outs, pos=used.expand(3, 11))


def test_strided_inputs_and_gradients():
    x = _inputs(2, 19, 4, 2, 128, 128, torch.bfloat16, seed=5)
    want, gwant = _both(x, False)
    y = dict(x)
    y["q"] = x["q"].transpose(1, 2).contiguous().transpose(1, 2)      # held as [B, H, S, D]
    y["k"] = x["k"].contiguous()
    got, ggot = _both(y, False)
    for a, b in zip(want + gwant, got + ggot):
        assert torch.equal(a, b)
    fused = torch.full((2, 19, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _, ggot = _both(x, False, dq=fused[:, :, :4], dk=fused[:, :, 4:6])
    assert torch.equal(fused[:, :, :4], gwant[0]) and torch.equal(fused[:, :, 4:6], gwant[1])
    assert bool((fused[:, :, 6:] == 7).all())


def test_inputs_shared_by_heads_and_batches():
    """Keys expanded over heads and queries over batches (strides of zero) are read in place;
    gradients come per head and batch."""
    x = _inputs(3, 7, 4, 4, 64, 64, torch.bfloat16, seed=15)
    x["k"] = x["k"][:, :, :1].expand(3, 7, 4, 64)
    x["q"] = x["q"][:1].expand(3, 7, 4, 64)
    outs, grads = _both(x, False)
    _check(x, 64, False, 1e-6, outs, grads)
    with pytest.raises(da.DashError) as e:
        _both(x, False, dq=torch.empty(1, 7, 4, 64, dtype=torch.bfloat16, device="cuda").expand(3, 7, 4, 64))
    assert e.value.status == da.DASH_ERR_INVALID_ARG


def test_empty():
    x = _inputs(2, 3, 4, 2, 64, 64, torch.bfloat16)
    e = lambda t: t[:, :0]
    a = (x["wq"], x["wk"], x["cos"], x["sin"])
    q, k = da.qk_norm_rope_forward(e(x["q"]), e(x["k"]), *a)
    assert q.shape == (2, 0, 4, 64) and k.shape == (2, 0, 2, 64)
    dq, dk, dwq, dwk = da.qk_norm_rope_backward(e(x["dq"]), e(x["dk"]), e(x["q"]), e(x["k"]), *a)
    assert float(dwq.abs().max()) == 0 and float(dwk.abs().max()) == 0


def test_zero_rows_with_eps():
    x = _inputs(1, 4, 2, 1, 64, 64, torch.float32, seed=6)
    x["q"] = torch.zeros_like(x["q"])
    outs, grads = _both(x, False, eps=1e-5)
    assert float(outs[0].abs().max()) == 0
    _check(x, 64, False, 1e-5, outs, grads)


def test_position_out_of_range():
    x = _inputs(1, 12, 2, 1, 64, 64, torch.bfloat16, P=30, seed=7)
    want, gwant = _both(x, False)
    x["pos"] = x["pos"].clone()
    x["pos"][0, 5] = 30
    x["pos"][0, 6] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"])
    outs = da.qk_norm_rope_forward(x["q"], x["k"], *a, status=status)
    assert int(status) == da.DASH_ERR_BOUNDS
    ws = da.new_qk_norm_rope_workspace(1, 12, 2, 1, 64, "cuda")
    grads = da.qk_norm_rope_backward(x["dq"], x["dk"], x["q"], x["k"], *a, workspace=ws, check=False)
    assert da.dash_attn_get_status(ws) == da.DASH_ERR_BOUNDS and "a position" in da.dash_last_error()
    keep = [0, 1, 2, 3, 4, 7, 8, 9, 10, 11]
    for got, w in zip(outs + grads[:2], want + gwant[:2]):
        assert bool(torch.isnan(got[:, 5:7]).all()) and torch.equal(got[:, keep], w[:, keep])


def test_bitwise_reproducible_streams_and_graph():
    x = _inputs(2, 700, 16, 4, 128, 64, torch.bfloat16, seed=8)
    ws = da.new_qk_norm_rope_workspace(2, 700, 16, 4, 128, "cuda")
    outs, grads = _both(x, True, workspace=ws)
    want = outs + grads
    for _ in range(5):
        ws.random_(0, 255)
        outs, grads = _both(x, True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, outs + grads))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs, grads = _both(x, True, workspace=ws, check=False)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs + grads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs, grads = _both(x, True, workspace=ws, check=False)
    for t in outs + grads:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs + grads))


def test_feeds_the_attention():
    """The outputs go straight into attn_forward; the gradients come straight back."""
    x = _inputs(1, 256, 2, 2, 64, 64, torch.bfloat16, seed=9)
    a = (x["wq"], x["wk"], x["cos"], x["sin"], x["pos"])
    q, k = da.qk_norm_rope_forward(x["q"], x["k"], *a)
    v = torch.randn_like(q)
    o, lse = da.attn_forward(q, k, v, 0.125, True)
    dq, dk, _ = da.attn_backward(q, k, v, o, torch.randn_like(o), lse, 0.125, True)
    x["dq"], x["dk"] = dq, dk
    _, grads = _both(x, False)
    _check(x, 64, False, 1e-6, None, grads)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hk,D,R", [(1, 4901, 27, 5, 64, 64), (2, 1361, 23, 6, 128, 64),
                                           (1, 3001, 23, 6, 96, 24), (1, 3001, 9, 4, 256, 20)])
def test_two_groups_of_heads_in_flight(t, il, B, S, Hq, Hk, D, R):
    """Rows enough that every warp of the forward handles two groups of heads at once (19456
    groups), with head counts that fill no group, all and part of the head rotated."""
    L = 4 if D <= 64 else 8 if D <= 128 else 16
    assert B * S * (Hq + Hk) // (2 * (32 // L)) >= 9728
    x = _inputs(B, S, Hq, Hk, D, R, t, seed=D + R)
    outs, grads = _both(x, il)
    _check(x, R, il, 1e-6, outs, grads)
    y = dict(x)
    y["q"] = x["q"].transpose(1, 2).contiguous().transpose(1, 2)
    got, _ = _both(y, il)
    assert all(torch.equal(a, b) for a, b in zip(outs, got))
