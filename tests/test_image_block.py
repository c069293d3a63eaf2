"""GPU: a block of a text-conditioned image model -- group norm, self attention with queries and
keys turned by two axes, cross attention to captions of unlike lengths -- run and differentiated
with the library's operators as a training step would, against float64 autograd of the formulas.

Every intermediate that the operators pass on is rounded to bf16 (2^-8 at most, 2^-9.6 in the mean
square); some ten of them lie between a parameter and its gradient, which in the mean square is
10^0.5 * 2^-9.6 = 0.4 %: held to 2 %. All results repeat in every bit."""
import math

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

B, H, W, C, HEADS, TXT, LENS = 2, 16, 16, 128, 2, 40, (40, 23)
D, S, SECTIONS = C // HEADS, H * W, (16, 16)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _data():
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    x = {"x": r(B, H, W, C), "text": r(B, TXT, 96), "dz": r(B, S, C, std=0.1)}
    for b, n in enumerate(LENS):
        x["text"][b, n:] = float("nan")              # what padding holds must not matter
    p = {"qkv": r(3 * C, C, std=C ** -0.5), "o": r(C, C, std=C ** -0.5), "cq": r(C, C, std=C ** -0.5),
         "ckv": r(2 * C, 96, std=96 ** -0.5), "co": r(C, C, std=C ** -0.5)}
    for n, d in (("gw", C), ("wq", D), ("wk", D)):
        p[n] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    p["gb"] = 0.1 * torch.randn(C, generator=g, device="cuda")
    i = torch.arange(S, device="cuda")
    pos = torch.stack([i // W, i % W])
    return x, p, pos, torch.tensor(LENS, device="cuda")


def _step(x, p, pos, lens):
    """Forward and backward with the operators; the gradients of the parameters, x and the text."""
    cos, sin = da.rope_axes_table(max(H, W), SECTIONS)
    rope = (p["wq"], p["wk"], cos, sin, pos, SECTIONS)
    scale = 1 / math.sqrt(D)
    h, mean, rstd = da.group_norm_act_forward(x["x"], p["gw"], p["gb"], 8)
    h = h.view(B * S, C)
    qkv = (h @ p["qkv"].t()).view(B, S, 3 * HEADS, D)
    q0, k0, v = qkv[:, :, :HEADS], qkv[:, :, HEADS:2 * HEADS], qkv[:, :, 2 * HEADS:].contiguous()
    q, k = da.qk_norm_rope_axes_forward(q0, k0, *rope)
    o, lse = da.attn_forward(q, k, v, scale, causal=False)
    y = x["x"].view(B * S, C) + o.view(B * S, C) @ p["o"].t()
    cq = (y @ p["cq"].t()).view(B, S, HEADS, D)
    ckv = (x["text"] @ p["ckv"].t()).view(B, TXT, 2 * HEADS, D)
    ck, cv = ckv[:, :, :HEADS], ckv[:, :, HEADS:]
    co, clse = da.cross_attn_forward(cq, ck, cv, scale, lens)
    z = y + co.view(B * S, C) @ p["co"].t()

    g = {}
    dz = x["dz"].view(B * S, C)
    g["co"] = dz.t() @ co.view(B * S, C)
    dco = (dz @ p["co"]).view(B, S, HEADS, D)
    dckv = torch.empty_like(ckv)
    dcq, _, _ = da.cross_attn_backward(cq, ck, cv, co, dco, clse, scale, lens, dk=dckv[:, :, :HEADS], dv=dckv[:, :, HEADS:])
    dcq, dckv = dcq.view(B * S, C), dckv.view(B * TXT, 2 * C)
    g["cq"] = dcq.t() @ y
    g["ckv"] = dckv.t() @ torch.nan_to_num(x["text"]).view(B * TXT, 96)
    g["text"] = dckv @ p["ckv"]
    dy = dz + dcq @ p["cq"]
    g["o"] = dy.t() @ o.view(B * S, C)
    do = (dy @ p["o"]).view(B, S, HEADS, D)
    dq, dk, dv = da.attn_backward(q, k, v, o, do, lse, scale, False, "shift", 1)
    dqkv = torch.empty_like(qkv)
    _, _, g["wq"], g["wk"] = da.qk_norm_rope_axes_backward(dq, dk, q0, k0, *rope, dq=dqkv[:, :, :HEADS],
                                                           dk=dqkv[:, :, HEADS:2 * HEADS])
    dqkv[:, :, 2 * HEADS:] = dv
    dqkv = dqkv.view(B * S, 3 * C)
    g["qkv"] = dqkv.t() @ h
    dh = (dqkv @ p["qkv"]).view(B, H, W, C)
    dx, g["gw"], g["gb"] = da.group_norm_act_backward(dh, x["x"], p["gw"], p["gb"], mean, rstd, 8)
    g["x"] = dx + dy.view(B, H, W, C)
    return z, g


def _formulas(x, p, pos):
    """The same in float64, differentiated by autograd."""
    p = {n: t.double().requires_grad_() for n, t in p.items()}
    xi = x["x"].double().requires_grad_()
    text = torch.nan_to_num(x["text"]).double().requires_grad_()
    cos, sin = (t.double() for t in da.rope_axes_table(max(H, W), SECTIONS))
    xg = xi.view(B, S, 8, C // 8)
    m = xg.mean((1, 3), keepdim=True)
    n = ((xg - m) / torch.sqrt(((xg - m) ** 2).mean((1, 3), keepdim=True) + 1e-5)).view(B, S, C) * p["gw"] + p["gb"]
    h = n * torch.sigmoid(n)
    q, k, v = (h @ p["qkv"].t()).view(B, S, 3, HEADS, D).unbind(2)
    axis = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(SECTIONS, device="cuda"))
    at = pos[axis].t()
    c, s = (t[at, torch.arange(D // 2, device="cuda")][None, :, None] for t in (cos, sin))

    def turn(t, w):
        t = t / torch.sqrt((t ** 2).mean(-1, keepdim=True) + 1e-6) * w
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def attend(q, k, v, lens):
        a = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
        hidden = torch.arange(k.shape[1], device="cuda")[None] >= torch.tensor(lens, device="cuda")[:, None]
        return torch.einsum("bhij,bjhd->bihd", a.masked_fill(hidden[:, None, None], -math.inf).softmax(-1), v)

    o = attend(turn(q, p["wq"]), turn(k, p["wk"]), v, (S, S)).reshape(B, S, C)
    y = xi.view(B, S, C) + o @ p["o"].t()
    cq = (y @ p["cq"].t()).view(B, S, HEADS, D)
    ck, cv = (text @ p["ckv"].t()).view(B, TXT, 2, HEADS, D).unbind(2)
    z = y + attend(cq, ck, cv, LENS).reshape(B, S, C) @ p["co"].t()
    (z * x["dz"].double()).sum().backward()
    g = {n: t.grad for n, t in p.items()}
    g["x"], g["text"] = xi.grad, text.grad
    return z.detach(), g


def test_block_matches_the_formulas_and_repeats():
    x, p, pos, lens = _data()
    z, g = _step(x, p, pos, lens)
    wz, wg = _formulas(x, p, pos)
    assert set(g) == set(wg)
    for name, got, want in [("z", z, wz)] + [(n, g[n], wg[n]) for n in g]:
        err = float((got.double().flatten() - want.flatten()).norm() / want.norm())
        assert err <= 2e-2, (name, err)
    for b, n in enumerate(LENS):
        assert not bool(g["text"].view(B, TXT, 96)[b, n:].any())
    z2, g2 = _step(x, p, pos, lens)
    assert torch.equal(z, z2) and all(torch.equal(g[n], g2[n]) for n in g)
