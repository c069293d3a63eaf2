"""CPU: the training-step operators' float64 oracle against central differences and small
hand-computed values."""
import math

import torch

from oracle import train_ops as ref

_g = torch.Generator().manual_seed(11)


def _randn(*shape):
    return torch.randn(*shape, generator=_g, dtype=torch.float64)


def _differences(f, x, h=1e-5):
    """Central differences of the scalar f at every element of x."""
    d = torch.zeros_like(x)
    for i in range(x.numel()):
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        d.view(-1)[i] = (f(a) - f(b)) / (2 * h)
    return d


def test_embed_gradient_matches_differences():
    table, ids, dout = _randn(7, 3), torch.tensor([2, 5, 2, 0, 6, 2]), _randn(6, 3)
    got = ref.embed_grad(dout, ids, 7, 1.7)
    want = _differences(lambda e: (dout * ref.embed(e, ids, 1.7)).sum(), table)
    assert torch.allclose(got, want, atol=1e-8)
    assert ref.embed_grad(dout, ids, 7, 1.7, padding_idx=2)[2].abs().max() == 0


def test_norm_rope_gradient_matches_differences():
    for interleaved in (False, True):
        x, w, d = _randn(2, 3, 2, 6), _randn(6), _randn(2, 3, 2, 6)
        ang = _randn(5, 2)
        cos, sin = ang.cos(), ang.sin()
        pos = torch.tensor([[0, 3, 4], [2, 2, 1]])
        f = lambda a, b: (d * ref.norm_rope(a, b, cos, sin, pos, 1e-3, interleaved)).sum()
        dx, dw = ref.norm_rope_grad(d, x, w, cos, sin, pos, 1e-3, interleaved)
        assert torch.allclose(dx, _differences(lambda a: f(a, w), x), atol=1e-7)
        assert torch.allclose(dw, _differences(lambda b: f(x, b), w), atol=1e-7)


def test_norm_rope_turns_a_known_vector():
    # one pair at 90 degrees: (a, b) -> (-b, a); the third and fourth columns pass
    x = torch.tensor([3.0, 4.0, 0.0, 0.0], dtype=torch.float64).view(1, 1, 1, 4)
    cos, sin = torch.zeros(1, 1, dtype=torch.float64), torch.ones(1, 1, dtype=torch.float64)
    y = ref.norm_rope(x, None, cos, sin, torch.zeros(1, 1, dtype=torch.long), 0.0, True).flatten()
    rms = math.sqrt(25 / 4)
    assert torch.allclose(y, torch.tensor([-4 / rms, 3 / rms, 0, 0], dtype=torch.float64))


def test_xent_gradient_matches_differences():
    x, w = _randn(4, 3), _randn(5, 3)
    y = torch.tensor([1, -100, 4, 0])
    dl = _randn(4)
    f = lambda a, b: (dl * ref.xent(a, b, y, -100, 0.7)[0]).sum()
    dx, dw, _, _ = ref.xent_grad(x, w, y, dl, -100, 0.7)
    assert torch.allclose(dx, _differences(lambda a: f(a, w), x), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda b: f(x, b), w), atol=1e-8)


def test_xent_of_equal_logits_is_log_v():
    loss, lse = ref.xent(torch.zeros(2, 3), torch.ones(8, 3), torch.tensor([0, -100]), -100)
    assert torch.allclose(lse, torch.full((2,), math.log(8), dtype=torch.float64))
    assert loss[1] == 0 and abs(loss[0] - math.log(8)) < 1e-12


def test_clip():
    norm, out = ref.clip([torch.tensor([3.0]), torch.tensor([4.0])], 1.0)
    assert abs(norm - 5) < 1e-12 and abs(out[0] - 0.6) < 1e-12 and abs(out[1] - 0.8) < 1e-12
    assert ref.clip([torch.tensor([3.0])], 4.0)[1][0] == 3.0
