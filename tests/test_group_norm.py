"""GPU: group norm with an activation, and its gradients, against the float64 definition.

Tolerances, with e = 2^-24. A thread sums every `lanes`-th row, at least 512 / C of them side by
side, then the lanes are joined in a few steps: a channel's sum of S values passes through at most
D = S min(C, 512) / 512 + 64 additions, each off by e of the sum of absolute values so far. The
mean is then off by dm = D e mean|x - K| and the variance by dv = 3 D e mean (x - K)^2 (K: the
channel's pivot; the factor for the square, its sum and the join), plus the 8 steps of what follows.
An fp32 z is off by 8 steps of its terms; the sigmoid by 2^-20 for |z| up to 30 (the exponent's
argument by |z| e); the activation's slope is at most 1.1 and its second derivative 0.5.
Gradients use the given mean and rstd; sums over N S rows: (D + N) e of the absolute values."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

TYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -140}
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(N, S, C, t, seed=0, mean=0.7, affine=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {"x": (r(N, S, C) * (1 + 0.5 * r(C).abs()) + mean * r(C)).to(t), "dy": r(N, S, C).to(t)}
    x["w"] = 1 + 0.2 * r(C) if affine else None
    x["b"] = 0.3 * r(C) if affine else None
    return x


def _depth(S, C):
    return S * min(C, 512) / 512 + 64


def _check_forward(x, G, eps, act, y, mean, rstd):
    xs = x["x"]
    N, S, C = xs.shape
    want, wm, wr = ref.group_norm(xs, x["w"], x["b"], G, eps, act)
    xh, z, r = ref._affine(xs, x["w"], x["b"], wm, wr, G)
    off = (xs.double() - xs[:, :1].double())
    per = lambda t: t.view(N, S, G, -1).mean((1, 3))  # noqa: E731
    D = _depth(S, C)
    dm = D * E * per(off.abs()) + 8 * E * wm.abs() + 8 * E * per(off ** 2).sqrt()
    dv = 3 * D * E * per(off ** 2) + dm ** 2
    dr = wr * (dv * wr ** 2 / 2 + 8 * E) * 1.01
    assert bool(((mean.double() - wm).abs() <= dm).all()), float(((mean.double() - wm).abs() - dm).max())
    assert bool(((rstd.double() - wr).abs() <= dr).all()), float(((rstd.double() - wr).abs() - dr).max())
    wide = lambda t: t.repeat_interleave(C // G, 1)[:, None]  # noqa: E731
    wa = torch.ones(C, device="cuda", dtype=torch.float64) if x["w"] is None else x["w"].double().abs()
    dxh = wide(dm) * r + xh.abs() * wide(dr / wr) + 8 * E * (xh.abs() + wide(wm.abs()) * r)
    dz = dxh * wa + 4 * E * (z.abs() + wa * xh.abs())
    u = torch.finfo(xs.dtype).eps / 2
    tol = (1.1 * dz + 2.0 ** -20 * z.abs()) * (1 + u) + u * want.abs() + TINY[xs.dtype]
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def _check_backward(x, G, act, mean, rstd, dx, dw, db):
    xs, dy = x["x"], x["dy"]
    N, S, C = xs.shape
    wdx, wdw, wdb, dz, xh = ref.group_norm_grad(dy, xs, x["w"], x["b"], mean, rstd, G, act)
    _, z, r = ref._affine(xs, x["w"], x["b"], mean, rstd, G)
    wa = torch.ones(C, device="cuda", dtype=torch.float64) if x["w"] is None else x["w"].double().abs()
    ma = mean.double().abs().repeat_interleave(C // G, 1)[:, None]
    dxh = 4 * E * (xh.abs() + (xs.double().abs() + ma) * r)
    dzz = 4 * E * (z.abs() + wa * xh.abs()) + dxh * wa
    # dz = dy act'(z): the sigmoid's error and z's
    ddz = dy.double().abs() * ((0.5 * dzz + 2.0 ** -20 * (1 + z.abs())) if act == "silu" else 0 * z) + 4 * E * dz.abs()
    D = _depth(S, C) + N
    ddb = (ddz + D * E * dz.abs()).sum((0, 1))
    ddw = (ddz * xh.abs() + dz.abs() * dxh + (D + 2) * E * (dz * xh).abs()).sum((0, 1))
    if x["w"] is not None:
        assert bool(((dw.double() - wdw).abs() <= ddw + 1e-38).all()), float(((dw.double() - wdw).abs() - ddw).max())
        assert bool(((db.double() - wdb).abs() <= ddb + 1e-38).all()), float(((db.double() - wdb).abs() - ddb).max())
    else:
        assert dw is None and db is None
    over = lambda t: t.view(N, S, G, -1).mean((1, 3)).repeat_interleave(C // G, 1)[:, None]  # noqa: E731
    D += C // G
    u1, u2 = (dz * wa).abs(), (dz * xh * wa).abs()
    e1 = over(ddz * wa + D * E * u1)
    e2 = over(ddz * xh.abs() * wa + dz.abs() * wa * dxh + (D + 4) * E * u2)
    tol = r * (ddz * wa + 8 * E * (u1 + over(u1) + xh.abs() * over(u2)) + e1 + xh.abs() * e2 + dxh * over(u2))
    u = torch.finfo(xs.dtype).eps / 2
    tol = tol * (1 + u) + u * wdx.abs() + TINY[xs.dtype]
    err = (dx.double() - wdx).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


SHAPES = [  # N, S, C, G
    (1, 1, 8, 1), (1, 1, 5, 5), (2, 64, 320, 32), (3, 1021, 250, 25), (2, 7, 6, 3), (1, 5000, 32, 4), (4, 33, 64, 64),
    (2, 100, 96, 1), (5, 30, 2048, 1), (1, 60000, 64, 4), (2, 20000, 24, 2), (3, 4096, 64, 32), (2, 11, 4096, 4),
    (1, 3, 9000, 3), (70, 2, 16, 2), (2, 9000, 128, 32)]


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,S,C,G", SHAPES)
def test_matches_definition(N, S, C, G, t, act):
    x = _inputs(N, S, C, t, seed=S + C)
    y, mean, rstd = da.group_norm_act_forward(x["x"], x["w"], x["b"], G, 1e-5, act)
    _check_forward(x, G, 1e-5, act, y, mean, rstd)
    grads = da.group_norm_act_backward(x["dy"], x["x"], x["w"], x["b"], mean, rstd, G, act)
    _check_backward(x, G, act, mean, rstd, *grads)


def _both(x, G, act="silu", **kw):
    y, mean, rstd = da.group_norm_act_forward(x["x"], x["w"], x["b"], G, 1e-5, act, **kw)
    return (y, mean, rstd, *da.group_norm_act_backward(x["dy"], x["x"], x["w"], x["b"], mean, rstd, G, act, **kw))


@pytest.mark.parametrize("t", TYPES)
def test_without_weights_and_with_one_of_them(t):
    x = _inputs(2, 50, 48, t, seed=1, affine=False)
    y, mean, rstd, *grads = _both(x, 6)
    _check_forward(x, 6, 1e-5, "silu", y, mean, rstd)
    _check_backward(x, 6, "silu", mean, rstd, *grads)
    w = torch.full((48,), 1.5, device="cuda")
    y, mean, rstd = da.group_norm_act_forward(x["x"], w, None, 6)
    dx, dw, db = da.group_norm_act_backward(x["dy"], x["x"], w, None, mean, rstd, 6)
    assert db is None and dw.shape == (48,)
    full = da.group_norm_act_backward(x["dy"], x["x"], w, torch.zeros(48, device="cuda"), mean, rstd, 6)
    assert torch.equal(dx, full[0]) and torch.equal(dw, full[1])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,S,C,G", [(2, 200, 64, 8), (1, 60000, 64, 4)])
def test_a_mean_far_beyond_the_spread(N, S, C, G, t):
    """Means a few hundred times the spread: in the first value's distance nothing is lost."""
    x = _inputs(N, S, C, t, seed=2, mean=0.0)
    x["x"] = (x["x"].float() + 100.0).to(t)
    y, mean, rstd, *grads = _both(x, G)
    _check_forward(x, G, 1e-5, "silu", y, mean, rstd)
    _check_backward(x, G, "silu", mean, rstd, *grads)


def test_constant_channels_and_large_activations():
    x = _inputs(2, 30, 32, torch.float32, seed=3)
    x["x"][:, :, :8] = 3.0                            # a group without spread
    x["b"][8:] = torch.linspace(-90, 90, 24, device="cuda")
    y, mean, rstd, *grads = _both(x, 4)
    assert bool(torch.isfinite(y).all()) and all(bool(torch.isfinite(g).all()) for g in grads)
    want, wm, wr = ref.group_norm(x["x"], x["w"], x["b"], 4, 1e-5, "silu")
    # the sigmoid's relative error at |z| <= 95: its exponent's argument is off by 2 steps of |z|
    tol = 2.0 ** -14 * want.abs() + 2.0 ** -16
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("t", TYPES)
def test_part_of_a_wider_buffer_and_maps(t):
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn(2, 6, 7, 96, generator=g, device="cuda").to(t)
    part = wide[..., 32:64]
    x = _inputs(2, 42, 32, t, seed=5)
    x["x"] = part.reshape(2, 42, 32)
    want = _both(x, 4)
    y = dict(x, x=part, dy=x["dy"].view(2, 6, 7, 32))
    got = _both(y, 4)
    assert got[0].shape == (2, 6, 7, 32)
    for a, b in zip(want, got):
        assert torch.equal(a.reshape(b.shape), b)
    odd = wide[..., 33:65]                            # no 16-byte pieces
    x["x"] = odd.reshape(2, 42, 32)
    y["x"] = odd
    got = _both(y, 4)
    _check_forward(x, 4, 1e-5, "silu", got[0].reshape(2, 42, 32), *got[1:3])
    with pytest.raises(ValueError, match="evenly"):
        da.group_norm_act_forward(wide[:, :, :5], None, None, 4)


def test_empty():
    for N, S in ((0, 5), (3, 0)):
        x = _inputs(N, S, 16, torch.bfloat16)
        y, mean, rstd, dx, dw, db = _both(x, 4)
        assert y.shape == (N, S, 16) and mean.shape == (N, 4)
        assert not bool(dw.any()) and not bool(db.any()) and not bool(mean.any())
        assert bool(torch.isfinite(rstd).all())


@pytest.mark.parametrize("N,S,C,G", [(2, 64, 320, 32), (4, 2000, 128, 8), (1, 60000, 64, 4)])
def test_bitwise_reproducible_streams_and_graph(N, S, C, G):
    x = _inputs(N, S, C, torch.bfloat16, seed=6)
    ws = da.new_group_norm_workspace(N, S, C, G, "cuda")
    want = _both(x, G, workspace=ws)
    for _ in range(5):
        ws.random_(0, 255)
        assert all(torch.equal(a, b) for a, b in zip(want, _both(x, G, workspace=ws)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _both(x, G)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    y, mean, rstd = da.group_norm_act_forward(x["x"], x["w"], x["b"], G, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _both(x, G, workspace=ws)
    for t in got:
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_given_outputs_and_refusals():
    x = _inputs(2, 10, 32, torch.bfloat16, seed=7)
    want = _both(x, 4)
    out, dx = torch.empty_like(x["x"]), torch.empty_like(x["x"])
    y, mean, rstd = da.group_norm_act_forward(x["x"], x["w"], x["b"], 4, out=out)
    assert y is out and torch.equal(out, want[0])
    got = da.group_norm_act_backward(x["dy"], x["x"], x["w"], x["b"], mean, rstd, 4, dx=dx)
    assert got[0] is dx and torch.equal(dx, want[3])
    bad = [dict(groups=5), dict(groups=0), dict(activation="relu"), dict(w=x["w"][:8]), dict(b=x["b"].double()),
           dict(x=x["x"].double()), dict(x=x["x"].transpose(1, 2))]
    for kw in bad:
        a = dict(dict(x=x["x"], w=x["w"], b=x["b"], groups=4, activation="silu"), **kw)
        with pytest.raises(ValueError):
            da.group_norm_act_forward(a["x"], a["w"], a["b"], a["groups"], activation=a["activation"])
    with pytest.raises(ValueError, match="dy"):
        da.group_norm_act_backward(x["dy"][:1], x["x"], x["w"], x["b"], mean, rstd, 4)
    with pytest.raises(ValueError, match="mean"):
        da.group_norm_act_backward(x["dy"], x["x"], x["w"], x["b"], mean[:, :2], rstd, 4)
    with pytest.raises(da.DashError) as e:
        da.group_norm_act_forward(x["x"], x["w"], x["b"], 4, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == da.DASH_ERR_WORKSPACE_TOO_SMALL
