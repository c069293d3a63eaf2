"""GPU: cross attention and its gradients against the float64 definition.

Tolerances, with u = 2^-8 the rounding of a bf16 value. Products of bf16 values are exact in
fp32 and the tensor core's fp32 additions are off by at most a step (2^-23) each, so a sum of n
products is off by at most n 2^-23 of the sum of their absolute values. A score over D values is
thus off by ez = (D + 16) 2^-23 scale sum |q k| (the 16 for the scaling, the subtraction and the
exponential, each at most a few steps of the score), and P by a factor of 1 + ez + 2^-19.
Forward: P is rounded to bf16 (u), O too; l sums the unrounded P.
Backward: P and dS are rounded to bf16 as operands; dP and Delta are sums of D products; what is
summed over n keys or rows is off by n 2^-23 more."""
import math

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(B, Sq, Sk, Hq, Hk, D, lens=None, seed=0, hide=True):
    """q, k and v as parts of projections, do; what lies behind a length is NaN and infinity."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    kv = randn(B, Sk, 2 * Hk, D)
    if lens is not None and hide:
        for b, n in enumerate(lens):
            kv[b, n:, 0::2] = float("nan")
            kv[b, n:, 1::2] = float("inf")
    x = {"q": randn(B, Sq, Hq + 1, D)[:, :, :Hq], "k": kv[:, :, :Hk], "v": kv[:, :, Hk:], "do": randn(B, Sq, Hq, D)}
    x["lens"] = [Sk] * B if lens is None else list(lens)
    x["t"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    x["scale"] = 1.0 / math.sqrt(D)
    return x


def _abs_products(a, b, lens, g):
    """sum |a| |b| over D for query rows a and key rows b, zero behind the lengths."""
    out = torch.zeros(a.shape[0], a.shape[2], a.shape[1], b.shape[1], dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n:
            out[i, :, :, :n] = a[i].double().abs().transpose(0, 1) @ ref._group(b[i:i + 1, :n], g)[0].abs().transpose(1, 2)
    return out


def _visible(x, lens):
    """A copy of [B, S, H, D] with zeros behind the lengths."""
    y = x.clone()
    for b, n in enumerate(lens):
        y[b, n:] = 0
    return y


def _check_forward(x, o, lse):
    q, k, v, lens = x["q"], x["k"], x["v"], x["lens"]
    D, g = q.shape[-1], q.shape[2] // k.shape[2]
    want, wlse, p = ref.cross_attn(q, k, v, lens, x["scale"])
    assert o.is_contiguous() and o.shape == q.shape and o.dtype == torch.bfloat16
    assert lse.shape == wlse.shape and lse.dtype == torch.float32
    ez = ((D + 16) * 2.0 ** -23 * x["scale"] * _abs_products(q, k, lens, g)).amax(-1) if k.shape[1] else 0 * wlse
    pv = (p @ ref._group(_visible(v, lens), g).abs()).transpose(1, 2)
    e = (2 * ez + 2.0 ** -18 + k.shape[1] * 2.0 ** -23).transpose(1, 2)[..., None]
    tol = (U + e) * pv + U * (1 + e) * want.abs() + 1e-38
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    none = torch.isinf(wlse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none) and not bool(torch.isnan(lse).any())
    tol = ez + (k.shape[1] / 32 + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + wlse.abs())
    assert bool(((lse.double() - wlse).abs() <= tol)[~none].all())


def _check_backward(x, o, lse, dq, dk, dv):
    q, k, v, do, lens, scale = (x[n] for n in ("q", "k", "v", "do", "lens", "scale"))
    B, Sq, Hq, D = q.shape
    Sk, Hk = k.shape[1], k.shape[2]
    g = Hq // Hk
    wq, wk, wv, p, ds = ref.cross_attn_grad(q, k, v, o, do, lse, lens, scale)
    lse0 = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).double().abs()[..., None]
    eP = (D + 16) * 2.0 ** -23 * scale * _abs_products(q, k, lens, g) + 2.0 ** -21 * (1 + lse0) + 2.0 ** -19
    delta = (do.double() * o.double()).abs().sum(-1).transpose(1, 2)[..., None]
    edp = (D + 16) * 2.0 ** -23 * (_abs_products(do, v, lens, g) + delta)
    eds = (U + eP) * ds.abs() + (1 + U) * p * edp                 # of dS as an operand
    n = lambda s: s * 2.0 ** -23  # noqa: E731
    kk = ref._group(_visible(k, lens), g).abs()
    shared = lambda t: t.view(B, Hk, g, Sk, D).sum(2).transpose(1, 2)  # noqa: E731
    qa, da_ = q.double().abs().transpose(1, 2), do.double().abs().transpose(1, 2)
    tq = scale * (((eds + n(Sk + 8) * ds.abs()) @ kk)).transpose(1, 2)
    tk = scale * shared((eds + n(Sq * g + 8) * ds.abs()).transpose(2, 3) @ qa)
    tv = shared(((U + eP + n(Sq * g + 8)) * p).transpose(2, 3) @ da_)
    for name, got, want, tol in (("dq", dq, wq, tq), ("dk", dk, wk, tk), ("dv", dv, wv, tv)):
        err = (got.double() - want).abs()
        tol = tol * (1 + U) + U * want.abs() + 1e-38
        assert bool((err <= tol).all()), (name, float((err - tol).max()))
    for b, m in enumerate(lens):
        assert not bool(dk[b, m:].any()) and not bool(dv[b, m:].any())
        assert m or not bool(dq[b].any())


SHAPES = [  # B, Sq, Sk, Hq, Hk, D, lens
    (1, 1, 1, 1, 1, 8, None), (2, 1, 77, 4, 4, 64, (77, 40)), (3, 5, 200, 8, 2, 128, (200, 0, 129)),
    (1, 130, 129, 2, 2, 64, None), (2, 300, 513, 4, 1, 128, (513, 385)), (1, 257, 1000, 6, 2, 80, (999,)),
    (7, 1, 1500, 8, 2, 128, (1500, 1, 700, 128, 0, 1024, 33)), (1, 64, 40, 5, 1, 40, None),
    (2, 129, 300, 3, 3, 96, (300, 256)), (1, 20, 260, 12, 2, 24, (257,)), (2, 70, 64, 1, 1, 16, (0, 0)),
    (4, 128, 128, 2, 1, 56, (128, 96, 95, 97)), (1, 400, 31, 3, 1, 128, (17,)), (1, 3, 4096, 2, 1, 64, None),
    (1, 2, 300, 200, 1, 32, None)]


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", SHAPES)
def test_forward_matches_definition(B, Sq, Sk, Hq, Hk, D, lens):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=Sq + Sk + D)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"], status=status)
    assert int(status) == 0
    _check_forward(x, o, lse)


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", SHAPES)
def test_backward_matches_definition(B, Sq, Sk, Hq, Hk, D, lens):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=Sq + Sk + D + 1)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    grads = da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"])
    _check_backward(x, o, lse, *grads)


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", [
    (4, 700, 77, 16, 16, 64, (77, 64, 30, 0)),        # more units than SMs, one key tile
    (3, 1500, 500, 8, 8, 128, (500, 129, 300)),       # several key tiles, the issuers take turns
    (2, 1100, 130, 12, 4, 96, (128, 130)), (1, 5000, 60, 1, 1, 128, None), (2, 1, 9000, 4, 4, 128, (9000, 4097))])
def test_more_units_than_multiprocessors(B, Sq, Sk, Hq, Hk, D, lens):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=Sq)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    _check_forward(x, o, lse)
    _check_backward(x, o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"]))


@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_grow_along_the_keys(D):
    """Scores from -40 to 40 in rising order, so that the exponent's reference moves at most key tiles."""
    x = _inputs(1, 200, 700, 2, 1, D, (650,), seed=3)
    q = torch.randn(1, 200, 1, D, device="cuda").sign()
    ramp = torch.linspace(-40, 40, 700, device="cuda")[None, :, None, None] / (D * x["scale"])
    x["q"] = q.expand(1, 200, 2, D).to(torch.bfloat16).contiguous()
    x["k"] = x["k"].clone()
    x["k"][:, :650] = (q[:, :1] * ramp[:, :650]).to(torch.bfloat16)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    _check_forward(x, o, lse)
    _check_backward(x, o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"]))


def test_strides_shared_batches_and_heads():
    x = _inputs(3, 70, 150, 4, 2, 64, (150, 20, 0), seed=5, hide=False)
    want = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    gwant = da.cross_attn_backward(x["q"], x["k"], x["v"], want[0], x["do"], want[1], x["scale"], x["t"])
    y = {n: x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"}          # held as [B, H, S, D]
    got = da.cross_attn_forward(y["q"], y["k"], y["v"], x["scale"], x["t"].long())
    fused = torch.full((3, 150, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dq = torch.full((3, 4, 70, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    ggot = da.cross_attn_backward(y["q"], y["k"], y["v"], got[0], x["do"], got[1], x["scale"], x["t"].long(), dq=dq,
                                  dk=fused[:, :, 1:3], dv=fused[:, :, 4:6])
    assert all(torch.equal(a, b) for a, b in zip(want + gwant, got + ggot))
    assert bool((fused[:, :, 0] == 7).all()) and bool((fused[:, :, 3] == 7).all())
    # keys of one batch and one head for all, queries of one head
    z = dict(x, k=x["k"][:1, :, :1].expand(3, 150, 2, 64), v=x["v"][:1, :, :1].expand(3, 150, 2, 64),
             q=x["q"][:, :, :1].expand(3, 70, 4, 64))
    o, lse = da.cross_attn_forward(z["q"], z["k"], z["v"], x["scale"], x["t"])
    _check_forward(z, o, lse)
    grads = da.cross_attn_backward(z["q"], z["k"], z["v"], o, x["do"], lse, x["scale"], x["t"])
    _check_backward(z, o, lse, *grads)
    with pytest.raises(da.DashError) as e:
        da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"], dk=z["k"])
    assert e.value.status == da.DASH_ERR_INVALID_ARG


def test_offsets_beyond_32_bits():
    """Keys of a batch that lies 2^32 elements behind the first one."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = _inputs(2, 9, 140, 2, 1, 64, (140, 135), seed=6, hide=False)
    flat = torch.empty((1 << 32) + 2 * 140 * 64, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((2, 140, 1, 64), (1 << 32, 64, 64, 1))
    far.copy_(x["k"])
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    want = (o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"]))
    got = da.cross_attn_forward(x["q"], far, x["v"], x["scale"], x["t"])
    dk = flat.as_strided((2, 140, 1, 64), (1 << 32, 64, 64, 1), 140 * 64)
    got = (*got, *da.cross_attn_backward(x["q"], far, x["v"], o, x["do"], lse, x["scale"], x["t"], dk=dk))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("Sq", [1, 200])
def test_length_out_of_range(Sq):
    x = _inputs(4, Sq, 300, 4, 2, 64, (300, 77, 20, 256), seed=7, hide=False)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    want = (o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"]))
    bad = x["t"].clone()
    bad[1], bad[2] = 301, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], bad, status=status)
    assert int(status) == da.DASH_ERR_BOUNDS
    ws = da.new_cross_attn_workspace(4, Sq, 300, 4, 2, 64, "cuda")
    got = (*got, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], bad, workspace=ws,
                                         check=False))
    assert da.dash_attn_get_status(ws) == da.DASH_ERR_BOUNDS and "a length" in da.dash_last_error()
    for a, b in zip(got, want):
        assert bool(torch.isnan(a[1:3]).all()) and torch.equal(a[0::3], b[0::3])
    with pytest.raises(da.DashError):
        da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], bad)


def test_empty():
    x = _inputs(2, 5, 40, 2, 2, 64, None, seed=8)
    none = x["k"][:, :0]
    o, lse = da.cross_attn_forward(x["q"], none, none, x["scale"])
    assert not bool(o.any()) and bool((lse == float("-inf")).all())
    dq, dk, dv = da.cross_attn_backward(x["q"], none, none, o, x["do"], lse, x["scale"])
    assert not bool(dq.any()) and dk.numel() == 0 and dv.numel() == 0
    q = x["q"][:, :0]
    o, lse = da.cross_attn_forward(q, x["k"], x["v"], x["scale"])
    assert o.shape == (2, 0, 2, 64) and lse.shape == (2, 2, 0)
    dq, dk, dv = da.cross_attn_backward(q, x["k"], x["v"], o, x["do"][:, :0], lse, x["scale"])
    assert dq.numel() == 0 and not bool(dk.any()) and not bool(dv.any())
    o, lse = da.cross_attn_forward(x["q"][:0], x["k"][:0], x["v"][:0], x["scale"])
    assert o.shape == (0, 5, 2, 64)


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", [
    (2, 300, 77, 4, 4, 64, (77, 50)), (3, 1, 1500, 8, 2, 128, (1500, 10, 700)), (2, 900, 400, 8, 4, 128, (400, 333))])
def test_bitwise_reproducible_streams_and_graph(B, Sq, Sk, Hq, Hk, D, lens):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=9)
    ws = da.new_cross_attn_workspace(B, Sq, Sk, Hq, Hk, D, "cuda")

    def both(**kw):
        o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"], workspace=ws)
        return (o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"],
                                                workspace=ws, **kw))
    want = both()
    for _ in range(5):
        ws.random_(0, 255)
        assert all(torch.equal(a, b) for a, b in zip(want, both()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both(check=False)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"], stream=s)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(check=False)
    for t in got:
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("Sq,Sk", [(300, 77), (300, 400)])
def test_a_wait_that_runs_out(Sq, Sk):
    """The testing hook withholds the tiles: every wait for them runs out, which the status and
    the LSE say; the next call is unharmed."""
    x = _inputs(1, Sq, Sk, 2, 2, 64, (Sk - 3,), seed=10)
    want = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        da.dash_debug_set_sync(50_000_000, 1)
        o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"], status=status)
        assert int(status) == da.DASH_ERR_SYNC_TIMEOUT and bool(torch.isnan(lse).all())
        with pytest.raises(da.DashError) as e:
            da.cross_attn_backward(x["q"], x["k"], x["v"], want[0], x["do"], want[1], x["scale"], x["t"])
        assert e.value.status == da.DASH_ERR_SYNC_TIMEOUT
    finally:
        da.dash_debug_set_sync(0, 0)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    _check_backward(x, o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"]))


def test_refusals():
    x = _inputs(2, 5, 40, 4, 2, 64, (40, 3), seed=11)
    f = lambda **kw: da.cross_attn_forward(*(dict(x, **kw)[n] for n in ("q", "k", "v", "scale", "t")))  # noqa: E731
    for kw in (dict(q=x["q"].float()), dict(k=x["k"][:, :, :1].expand(2, 40, 3, 64)), dict(v=x["v"][:, :39]),
               dict(t=x["t"].float()), dict(t=x["t"][:1]), dict(q=x["q"][:1]), dict(q=x["q"].transpose(2, 3))):
        with pytest.raises(ValueError):
            f(**kw)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(da.DashError) as e:
            f(**kw)
        assert e.value.status == da.DASH_ERR_INVALID_ARG
    o, lse = f()
    b = lambda **kw: da.cross_attn_backward(*(dict(x, o=o, lse=lse, **kw)[n] for n in  # noqa: E731
                                              ("q", "k", "v", "o", "do", "lse", "scale", "t")))
    for kw in (dict(do=x["do"].transpose(1, 2).contiguous().transpose(1, 2)), dict(do=x["do"][:, :4])):
        with pytest.raises(ValueError):
            b(**kw)
    with pytest.raises(ValueError):
        da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse[:, :, :4], x["scale"], x["t"])
    with pytest.raises(da.DashError) as e:
        da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"],
                               workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == da.DASH_ERR_WORKSPACE_TOO_SMALL
