"""CPU: the float64 definitions of cross attention, the rotation over several axes and the group
norm against central differences and small hand-computed values."""
import math

import torch

from oracle import train_ops as ref
from tests.test_train_oracle import _differences, _randn


def test_cross_attention_by_hand():
    q = torch.zeros(2, 1, 2, 3, dtype=torch.float64)
    k, v = _randn(2, 4, 1, 3), _randn(2, 4, 1, 3)
    o, lse, p = ref.cross_attn(q, k, v, [3, 0], 0.5)
    assert torch.allclose(o[0, 0, 0], v[0, :3, 0].mean(0)) and torch.allclose(o[0, 0, 1], v[0, :3, 0].mean(0))
    assert torch.allclose(lse[0], torch.full((2, 1), math.log(3), dtype=torch.float64))
    assert not o[1].any() and bool((lse[1] == -math.inf).all()) and not p[1].any() and not p[0, :, :, 3].any()


def test_cross_attention_gradient_matches_differences():
    q, k, v, do, lens = _randn(2, 3, 4, 3), _randn(2, 5, 2, 3), _randn(2, 5, 2, 3), _randn(2, 3, 4, 3), [4, 2]
    loss = lambda q, k, v: (do * ref.cross_attn(q, k, v, lens, 0.7)[0]).sum()  # noqa: E731
    o, lse, _ = ref.cross_attn(q, k, v, lens, 0.7)
    dq, dk, dv, _, _ = ref.cross_attn_grad(q, k, v, o, do, lse, lens, 0.7)
    assert torch.allclose(dq, _differences(lambda t: loss(t, k, v), q), atol=1e-8)
    assert torch.allclose(dk, _differences(lambda t: loss(q, t, v), k), atol=1e-8)
    assert torch.allclose(dv, _differences(lambda t: loss(q, k, t), v), atol=1e-8)


def test_axes_gradient_matches_differences():
    for il in (False, True):
        x, w, d = _randn(2, 3, 2, 8), _randn(8), _randn(2, 3, 2, 8)
        ang = _randn(5, 3)
        pos = torch.tensor([[[0, 3, 4], [2, 2, 1]], [[1, 1, 0], [4, 3, 2]]])
        args = (ang.cos(), ang.sin(), pos, (1, 2), 1e-3, il)
        y = ref.norm_rope_axes(x, w, *args)
        # pair 1 belongs to axis 1: token (0, 0) turns it by the angle of position 1, column 1
        n = x[0, 0, 0] / torch.sqrt((x[0, 0, 0] ** 2).mean() + 1e-3) * w
        a, b = (2, 3) if il else (1, 4)
        c, s = ang[1, 1].cos(), ang[1, 1].sin()
        assert torch.allclose(y[0, 0, 0, a], n[a] * c - n[b] * s) and torch.allclose(y[0, 0, 0, b], n[b] * c + n[a] * s)
        dx, dw = ref.norm_rope_axes_grad(d, x, w, *args)
        assert torch.allclose(dx, _differences(lambda t: (d * ref.norm_rope_axes(t, w, *args)).sum(), x), atol=1e-7)
        assert torch.allclose(dw, _differences(lambda t: (d * ref.norm_rope_axes(x, t, *args)).sum(), w), atol=1e-7)


def test_group_norm_gradient_matches_differences():
    for act in ("none", "silu"):
        x, w, b, dy = _randn(2, 3, 6), _randn(6), _randn(6), _randn(2, 3, 6)
        f = lambda x, w, b: (dy * ref.group_norm(x, w, b, 2, 1e-3, act)[0]).sum()  # noqa: E731
        y, mean, rstd = ref.group_norm(x, w, b, 2, 1e-3, act)
        assert torch.allclose(mean[1, 1], x[1, :, 3:].mean())
        assert torch.allclose(rstd[1, 1], (x[1, :, 3:].var(unbiased=False) + 1e-3).rsqrt())
        dx, dw, db, _, _ = ref.group_norm_grad(dy, x, w, b, mean, rstd, 2, act)
        assert torch.allclose(dx, _differences(lambda t: f(t, w, b), x), atol=1e-7)
        assert torch.allclose(dw, _differences(lambda t: f(x, t, b), w), atol=1e-7)
        assert torch.allclose(db, _differences(lambda t: f(x, w, t), b), atol=1e-7)
