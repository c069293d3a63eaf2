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
