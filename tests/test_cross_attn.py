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
