"""GPU: group norm at the edges of what it accepts, against the float64 definition."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

TYPES = [torch.bfloat16, torch.float16, torch.float32]
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("C,G", [(1024, 1), (2048, 1), (4096, 1), (8192, 2), (1026, 2)])
def test_no_rows_with_wide_groups(C, G, t):
    """Groups of more channels than a block has threads, and no row to take a value from."""
    x = torch.empty(3, 0, C, dtype=t, device="cuda")
    w, b = torch.rand(C, device="cuda"), torch.rand(C, device="cuda")
    y, mean, rstd = da.group_norm_act_forward(x, w, b, G, 0.25)
    assert y.shape == x.shape and not bool(mean.any()) and bool(((rstd - 2).abs() <= 8 * E).all())
    dx, dw, db = da.group_norm_act_backward(x, x, w, b, mean, rstd, G)
    assert dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())


def _sums(xs, G):
    N, S, C = xs.shape
    return lambda t: t.view(N, -1, G, C // G).mean((1, 3))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("mean", [0.0, 100.0, 1000.0])
@pytest.mark.parametrize("where", [0, -1, "half"])
@pytest.mark.parametrize("N,S,C,G", [(2, 65536, 64, 4), (1, 1 << 20, 16, 1), (1, 65536, 25, 5), (4, 4096, 128, 8),
                                     (2, 300, 48, 3), (3, 7, 64, 4)])
def test_a_row_unlike_the_others(N, S, C, G, where, mean, t):
    """One row (the first, the last or the middle one) of zeros, or 300 spreads away where the mean
    is 0. A channel's sums are taken around the median of five of its values, so at most one of five
    is far off and |K - m| <= 3 s, with m and s the channel's mean and spread without that row (three
    of five normal values beyond 3 s: 5e-8). At these sizes a value passes through at most 128 additions
    (a thread's rows, the block's lanes, the chunks), each off by e: the mean is off by
    dm = 128 e (mean |x - m| + 3 s), the variance by 3 * 128 e (mean (x - m)^2 + 9 s^2)."""
    g = torch.Generator(device="cuda").manual_seed(S + C)
    x = (torch.randn(N, S, C, generator=g, device="cuda") + mean).to(t)
    at = S // 2 if where == "half" else where
    x[:, at] = 0.0 if mean else 300.0
    y, mu, rstd = da.group_norm_act_forward(x, None, None, G, 1e-5, "none")
    want, wm, wr = ref.group_norm(x, None, None, G, 1e-5, "none")
    xd = x.double()
    rest = torch.cat((xd[:, :at % S], xd[:, at % S + 1:]), 1)
    m, s = rest.mean(1, keepdim=True), rest.std(1, keepdim=True)
    per = _sums(x, G)
    dm = 128 * E * (per((xd - m).abs()) + per(3 * s)) + 2 * E * wm.abs()
    dv = 3 * 128 * E * (per((xd - m) ** 2) + per(9 * s ** 2))
    dr = wr * (dv * wr ** 2 / 2 + 8 * E) * 1.01
    assert bool(((mu.double() - wm).abs() <= dm).all()), float(((mu.double() - wm).abs() / dm).max())
    assert bool(((rstd.double() - wr).abs() <= dr).all()), float(((rstd.double() - wr).abs() / dr).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,S,C,G", [(2, 64, 64, 4), (1, 20000, 64, 4), (1, 20000, 24, 8), (2, 50, 25, 5)])
def test_groups_of_one_value(N, S, C, G, t):
    """x - mean is 0, so y is act(b) whatever the size of the mean and of rstd; dx has no part along xh."""
    g = torch.Generator(device="cuda").manual_seed(3)
    v = torch.tensor([1000.0, -640.0, 3.0, 0.0], device="cuda").repeat(8)[:G].repeat_interleave(C // G)
    x = v.to(t).expand(N, S, C).contiguous()
    w, b = torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    u = torch.finfo(t).eps / 2
    for act in ("none", "silu"):
        y, mean, rstd = da.group_norm_act_forward(x, w, b, G, 1e-5, act)
        want, wm, wr = ref.group_norm(x, w, b, G, 1e-5, act)
        assert torch.equal(mean.double(), wm)
        err = (y.double() - want).abs()
        assert bool((err <= (u + 2.0 ** -20) * want.abs() + 2.0 ** -25).all()), float(err.max())


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("N,S,C,G", [(2, 64, 64, 4), (1, 20000, 64, 4), (1, 20000, 24, 8), (2, 50, 25, 5)])
def test_gradient_far_from_zero(N, S, C, G, act):
    """fp32 values within a factor of two of the given mean: x - mean is exact, so nothing of the mean's
    size is in the gradients' errors. z is off by 4 steps of its terms, the sigmoid and its slope by
    2^-20 (1 + |z|); the group's means are sums of n = S C / G values that pass through at most 256
    additions here."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(N, S, C, generator=g, device="cuda") + 1000.0
    dy = torch.randn(N, S, C, generator=g, device="cuda")
    w, b = 1 + 0.2 * torch.randn(C, generator=g, device="cuda"), 0.3 * torch.randn(C, generator=g, device="cuda")
    _, mean, rstd = da.group_norm_act_forward(x, w, b, G, 1e-5, act)
    dx, dw, db = da.group_norm_act_backward(dy, x, w, b, mean, rstd, G, act)
    wdx, wdw, wdb, dz, xh = ref.group_norm_grad(dy, x, w, b, mean, rstd, G, act)
    _, z, r = ref._affine(x, w, b, mean, rstd, G)
    wa = w.double().abs()
    ez = 4 * E * (z.abs() + wa * xh.abs() + b.double().abs())
    ddz = dy.double().abs() * ((0.5 * ez + 2.0 ** -20 * (1 + z.abs())) if act == "silu" else 0 * z) + 4 * E * dz.abs()
    over = lambda t: _sums(x, G)(t).repeat_interleave(C // G, 1)[:, None]  # noqa: E731
    u1, u2 = (dz * wa).abs(), (dz * xh * wa).abs()
    e1, e2 = over(ddz * wa + 256 * E * u1), over(ddz * xh.abs() * wa + 260 * E * u2)
    tol = r * (ddz * wa + e1 + xh.abs() * e2 + 8 * E * (u1 + over(u1) + xh.abs() * over(u2)))
    err = (dx.double() - wdx).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    ddw = (ddz * xh.abs() + 260 * E * (dz * xh).abs()).sum((0, 1))
    assert bool(((dw.double() - wdw).abs() <= ddw).all())
    assert bool(((db.double() - wdb).abs() <= (ddz + 256 * E * dz.abs()).sum((0, 1))).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,S,C,G", [(2, 64, 320, 32), (4, 2000, 128, 8), (4, 4096, 512, 32), (1, 60000, 64, 4), (3, 50, 25, 5)])
def test_in_place(N, S, C, G, t):
    """y over x, and dx over x or over dy: the bits of the call with an output of its own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(N, S, C, generator=g, device="cuda").to(t)
    dy = torch.randn(N, S, C, generator=g, device="cuda").to(t)
    w, b = torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    want = da.group_norm_act_forward(x, w, b, G)
    grads = da.group_norm_act_backward(dy, x, w, b, *want[1:], G)
    for _ in range(3):
        y = x.clone()
        got = da.group_norm_act_forward(y, w, b, G, out=y)
        assert got[0] is y and all(torch.equal(p, q) for p, q in zip(got, want))
        for over in (0, 1):
            a = [x.clone(), dy.clone()]
            got = da.group_norm_act_backward(a[1], a[0], w, b, *want[1:], G, dx=a[over])
            assert got[0] is a[over] and all(torch.equal(p, q) for p, q in zip(got, grads))


def test_outputs_that_overlap_otherwise_are_refused():
    flat = torch.randn(4000, device="cuda")
    x, w = flat[:3200].view(2, 50, 32), torch.ones(32, device="cuda")
    _, mean, rstd = da.group_norm_act_forward(x, w, None, 4)
    shifted, wide = flat[32:3232].view(2, 50, 32), flat[:3840].view(2, 60, 32)[:, :50]
    part = flat[:3200].view(2, 25, 64)[..., :32]
    for y, out in ((x, shifted), (shifted, x), (wide, x), (part, flat[:1600].view(2, 25, 32))):
        with pytest.raises(ValueError, match="overlap"):
            da.group_norm_act_forward(y, w, None, 4, out=out)
    dy = torch.randn_like(x)
    with pytest.raises(ValueError, match="overlap"):
        da.group_norm_act_backward(dy, x, w, None, mean, rstd, 4, dx=shifted)
    with pytest.raises(ValueError, match="overlap"):
        da.group_norm_act_backward(shifted, dy, w, None, mean, rstd, 4, dx=x)


def test_gradient_without_rows_and_eps():
    """rstd is infinite, the sums over no row are 0 all the same."""
    x = torch.empty(2, 0, 32, device="cuda")
    w, b = torch.rand(32, device="cuda"), torch.rand(32, device="cuda")
    y, mean, rstd = da.group_norm_act_forward(x, w, b, 4, 0.0)
    assert bool(torch.isinf(rstd).all())
    dx, dw, db = da.group_norm_act_backward(x, x, w, b, mean, rstd, 4)
    assert not bool(dw.any()) and not bool(db.any())
