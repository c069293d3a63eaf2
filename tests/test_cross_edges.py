"""GPU: cross attention at the edges of what it accepts: scores of minus infinity, gradients that are
not finite, long states."""
import math

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built, has_gpu
from tests.test_cross_attn import _check_forward, _inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,n", [
    (1, 300, 700, 2, 1, 64, 130), (1, 300, 700, 2, 1, 128, 130), (2, 1, 1500, 8, 2, 128, 900),
    (1, 2000, 400, 16, 16, 64, 256), (1, 2000, 400, 16, 16, 128, 257), (3, 40, 90, 4, 2, 80, 89), (1, 1, 9000, 1, 1, 64, 8999)])
def test_leading_scores_of_minus_infinity(B, Sq, Sk, Hq, Hk, D, n):
    """The first n keys have a score of -inf with every query: their weight is 0, whatever the other
    key tiles and ranges hold."""
    x = _inputs(B, Sq, Sk, Hq, Hk, D, None, seed=n)
    x["q"], x["k"] = x["q"].clone(), x["k"].clone()
    x["q"][..., 3] = x["q"][..., 3].abs() + 0.5
    x["k"][:, :n, :, 3] = -INF
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"])
    y = dict(x, k=x["k"][:, n:], v=x["v"][:, n:], lens=[Sk - n] * B)
    _check_forward(y, o, lse)


@pytest.mark.parametrize("Sq,Sk,Hq,D", [(128, 77, 2, 64), (256, 300, 2, 128), (2048, 300, 16, 64), (1, 1500, 4, 128)])
def test_rows_whose_scores_are_all_minus_infinity(Sq, Sk, Hq, D):
    """They see no key: O = 0 and LSE = -inf, as with a length of 0, and no gradient reaches v from them."""
    x = _inputs(1, Sq, Sk, Hq, Hq, D, None, seed=Sk)
    q, k, v, do = x["q"].clone(), x["k"].clone(), x["v"], x["do"]
    q[..., 3] = 0.5 + q[..., 3].abs()
    k[:, :, 0, 3] = -INF                              # head 0
    o, lse = da.cross_attn_forward(q, k, v, x["scale"])
    assert not bool(o[:, :, 0].any()) and bool((lse[:, 0] == -INF).all())
    some = lambda t: t[:, :, 1:]  # noqa: E731
    _check_forward(dict(x, q=some(q), k=some(k), v=some(v)), some(o).contiguous(), lse[:, 1:])
    dq, dk, dv = da.cross_attn_backward(q, k, v, o, do, lse, x["scale"])
    assert Sq == 1 or not bool(dv[:, :, 0].any())
    assert all(bool(torch.isfinite(t[:, :, 1:]).all()) for t in (dq, dk, dv))


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", [
    (1, 130, 77, 2, 2, 64, None), (1, 130, 300, 2, 1, 128, None), (2, 40, 90, 6, 2, 128, (90, 80)),
    (3, 1, 1500, 8, 2, 64, (1500, 700, 900)), (1, 1000, 500, 16, 16, 64, None), (1, 200, 60, 3, 1, 128, None)])
def test_places_of_a_row_tile_without_a_row(B, Sq, Sk, Hq, Hk, D, lens):
    """Keys whose scores are -inf with every query weigh 0 and get no gradient; nor may the places behind a
    tile's last row give them one (zeros times an infinite key). The others' gradients are those of the call
    without such keys."""
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=Sq, hide=False)
    x["q"] = x["q"].clone()
    x["q"][..., 3] = 0.5 + x["q"][..., 3].abs()
    k = x["k"].clone()
    k[:, 5::7, :, 3] = -INF
    o, lse = da.cross_attn_forward(x["q"], k, x["v"], x["scale"], x["t"])
    _, dk, dv = da.cross_attn_backward(x["q"], k, x["v"], o, x["do"], lse, x["scale"], x["t"])
    assert not bool(dk[:, 5::7].any()) and not bool(dv[:, 5::7].any())
    _, dk0, dv0 = da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"])
    keep = torch.arange(Sk, device="cuda") % 7 != 5
    assert torch.equal(dk[:, keep], dk0[:, keep]) and torch.equal(dv[:, keep], dv0[:, keep])


@pytest.mark.parametrize("bad", [float("nan"), INF])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", [
    (2, 300, 77, 4, 2, 64, (50, 77)), (2, 300, 77, 4, 2, 128, (50, 0)), (2, 300, 513, 4, 1, 128, (400, 257)),
    (1, 1, 1500, 4, 4, 64, (700,)), (1, 5000, 60, 1, 1, 128, (33,))])
def test_rows_behind_a_length_are_zero_whatever_the_gradient(B, Sq, Sk, Hq, Hk, D, lens, bad):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=12)
    o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"])
    do = x["do"].clone()
    do[:, Sq // 2, Hq - 1, D // 2] = bad
    dq, dk, dv = da.cross_attn_backward(x["q"], x["k"], x["v"], o, do, lse, x["scale"], x["t"])
    for b, m in enumerate(lens):
        assert not bool(dk[b, m:].any()) and not bool(dv[b, m:].any())
        assert m == 0 or not bool(torch.isfinite(dv[b, :m, Hk - 1, D // 2]).any())


def _same_rows(Sq, Sk, H, seed):
    """Queries that are all alike, so that one row says what each is: scores of any sign, values and a key
    column whose products with dS have one sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sign = (torch.randint(0, 2, (Sk,), generator=g, device="cuda") * 2 - 1).bfloat16()
    k = torch.zeros(1, Sk, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, :, 0, 0] = torch.randn(Sk, generator=g, device="cuda").bfloat16()
    k[0, :, 0, 1] = sign                               # the queries' column 1 is 0
    v[0, :, 0, 0] = sign
    v[0, :, 0, 1] = 1.0
    q = torch.zeros(1, Sq, H, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    do = torch.zeros_like(q)
    do[..., 0] = 1.0
    return q, k, v, do


@pytest.mark.parametrize("Sk", [1 << 16, (1 << 16) + 1, (1 << 21) + 77, 1 << 22])
def test_long_states(Sk):
    """Sums of one sign over millions of keys. The tensor core truncates: each of the n / 16 additions of
    a unit loses up to two steps (2^-23) of the sum so far, half the last one on average, n 2^-27 in all, 2^-11
    over the 65536 keys that a unit takes at most; beside the roundings of P or dS (2^-8 of each, which average:
    8 times 2^-8 / sqrt(n)) and of the result."""
    H, Sq = 1, 77 * 256
    q, k, v, do = _same_rows(Sq, Sk, H, seed=Sk)
    o, lse = da.cross_attn_forward(q, k, v, 1.0)
    z = k[0, :, 0, 0].double()
    s = v[0, :, 0, 0].double()
    p = torch.softmax(z, 0)
    u = 2.0 ** -8
    tol = 2.0 ** -11 + u / math.sqrt(Sk) * 8 + 2.0 ** -20
    assert bool(((lse.double() - torch.logsumexp(z, 0)).abs() <= 2.0 ** -16).all())
    # (a bf16 value just below 1 is off by at most 2^-9)
    assert bool(((o[..., 1].double() - 1).abs() <= u / 2 + tol).all()), float(o[..., 1].float().min())
    want = float((p * s).sum())
    assert bool(((o[..., 0].double() - want).abs() <= u * abs(want) + tol).all())
    # dS = P (s - delta), dQ's column 1 = sum dS s, of one sign
    delta = o[0, 0, 0, 0].double()
    dq, dk, dv = da.cross_attn_backward(q, k, v, o, do, lse, 1.0)
    want = float((torch.exp(z - lse[0, 0, 0].double()) * (s - delta) * s).sum())
    assert bool(((dq[..., 1].double() - want).abs() <= (u / 2 + tol) * abs(want) + 2.0 ** -20).all()), (
        float(dq[..., 1].float().min()), want)


def test_no_batch_with_a_workspace():
    ws = da.new_cross_attn_workspace(0, 5, 40, 2, 1, 64, "cuda")
    q, k = torch.empty(0, 5, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 40, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = da.cross_attn_forward(q, k, k, 1.0, workspace=ws)
    grads = da.cross_attn_backward(q, k, k, o, q, lse, 1.0, workspace=ws)
    assert o.shape == q.shape and [t.shape for t in grads] == [q.shape, k.shape, k.shape]
    assert da.dash_attn_get_status(ws) == da.DASH_OK
