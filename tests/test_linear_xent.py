"""GPU: cross entropy from hidden states and its gradient against the float64 definition.

Tolerances, element by element, from the roundings on the way (u = 2^-8, half a step of bf16):
* a logit: D products, exact in fp32, summed in fp32 in any order with truncation at worst:
  ez = D 2^-23 max_v sum_i |x_i w_vi| scale, plus the two roundings of its scaling;
* lse, loss: ez + the exponentials (2^-21 relative) + the sums (at most 64 serial additions a
  half tile, the joins of the half tiles: 2^-24 each, at most 2^10 of them) + its own rounding;
* G: u |G| for its rounding to bf16 (u^2 up to 128 tokens, where it is held as two terms), and
  g p (2 ez + 2^-20) for the logit and lse in it;
* dX, dW: those through the absolute products, fp32 sums (K 2^-23), u of the result.
"""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

U = 2.0 ** -8
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(T, V, D, seed=0, idt=torch.int64, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(V, D, generator=g, device="cuda").mul_(1.5 / D ** 0.5).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, D, generator=g, device="cuda") + 4 * torch.rand(T, 1, generator=g, device="cuda") * w[y].float()
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, torch.full_like(y, IGN), y)
    dl = torch.randn(T, generator=g, device="cuda") / max(T, 1)
    return x.bfloat16(), w, y.to(idt), dl


def _check(x, w, y, dl, loss, lse, dx=None, dw=None, scale=1.0, base=None):
    T, D = x.shape
    xd, wd = x.double().abs(), w.double().abs()
    loss64, lse64 = ref.xent(x, w, y, IGN, scale)
    ez = (D * 2.0 ** -23 + 2.0 ** -22) * scale * (xd @ wd.t()).amax(1)
    tol = 2 * ez + 2.0 ** -21 + 2.0 ** -14 + 2.0 ** -23 * lse64.abs()
    assert bool(((lse.double() - lse64).abs() <= tol).all())
    assert bool(((loss.double() - loss64).abs() <= 2 * tol).all())
    assert bool((loss[y == IGN] == 0).all())
    if dx is None:
        return
    dx64, dw64, G, gp = ref.xent_grad(x, w, y, dl, IGN, scale)
    eG = (U if T > 128 else U * U) * G.abs() + gp * (tol[:, None] + ez[:, None] + 2.0 ** -20)
    V = w.shape[0]
    bx = eG @ wd + V * 2.0 ** -23 * (G.abs() @ wd) + U * dx64.abs() + 1e-30
    assert bool(((dx.double() - dx64).abs() <= bx).all()), float(((dx.double() - dx64).abs() / bx).max())
    udw = U if dw.dtype == torch.bfloat16 else 2.0 ** -24
    if base is not None:
        dw64 = dw64 + base.double()
    bw = eG.t() @ xd + T * 2.0 ** -23 * (G.abs().t() @ xd) + udw * dw64.abs() * 1.01 + 1e-30
    assert bool(((dw.double() - dw64).abs() <= bw).all()), float(((dw.double() - dw64).abs() / bw).max())


@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (1, 300, 64), (2, 7, 72), (127, 255, 64), (128, 256, 128),
                                   (129, 257, 136), (300, 1000, 512), (333, 5003, 1024), (17, 20011, 264),
                                   (2500, 700, 320)])
def test_matches_definition(T, V, D):
    x, w, y, dl = _inputs(T, V, D, seed=T + V)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("dwt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types_scale_and_accumulation(idt, dwt, accumulate):
    T, V, D = 200, 999, 200
    x, w, y, dl = _inputs(T, V, D, seed=5, idt=idt)
    loss, lse = da.linear_xent_forward(x, w, y, scale=0.37)
    base = torch.randn(V, D, device="cuda").mul_(1e-2).to(dwt) if accumulate else None
    dw = base.clone() if accumulate else torch.full((V, D), float("nan"), dtype=dwt, device="cuda")
    dx, out = da.linear_xent_backward(x, w, y, lse, dl, scale=0.37, dw=dw, accumulate=accumulate)
    assert out is dw
    _check(x, w, y.long(), dl, loss, lse, dx, dw, 0.37, base)


def test_several_pieces_of_the_vocabulary():
    """T * V large enough that G does not fit one piece of the workspace."""
    T, V, D = 4096, 70001, 64
    x, w, y, dl = _inputs(T, V, D, seed=6)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


def test_several_pieces_with_split_ranges():
    T, V, D = 300, 500000, 8
    x, w, y, dl = _inputs(T, V, D, seed=7)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


@pytest.mark.parametrize("T,V,D", [(64, 40000, 1024), (1300, 20000, 2048)])
def test_products_of_many_tiles(T, V, D):
    """dX and dW in launches of their own (few tiles share one), dX split over K and not."""
    x, w, y, dl = _inputs(T, V, D, seed=T)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


def test_row_strides():
    T, V, D = 130, 300, 64
    x, w, y, dl = _inputs(T, V, D, seed=8)
    xs = torch.full((T, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 8:8 + D]
    ws = torch.full((V, 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda")[:, D:]
    xs.copy_(x)
    ws.copy_(w)
    loss, lse = da.linear_xent_forward(x, w, y)
    loss2, lse2 = da.linear_xent_forward(xs, ws, y)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    for a, b in zip(da.linear_xent_backward(x, w, y, lse, dl), da.linear_xent_backward(xs, ws, y, lse, dl)):
        assert torch.equal(a, b)


def test_all_rows_ignored_and_no_rows():
    x, w, y, dl = _inputs(50, 300, 64, seed=9, ignored=2.0)
    loss, lse = da.linear_xent_forward(x, w, y)
    assert float(loss.abs().max()) == 0 and bool(torch.isfinite(lse).all())
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    assert float(dx.abs().max()) == 0 and float(dw.abs().max()) == 0
    loss, lse = da.linear_xent_forward(x[:0], w, y[:0])
    assert loss.shape == (0,)
    dw = torch.full((300, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx, _ = da.linear_xent_backward(x[:0], w, y[:0], lse, dl[:0], dw=dw)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0


def test_nan_and_inf_stay_in_their_rows():
    x, w, y, dl = _inputs(140, 300, 64, seed=10, ignored=0.0)
    want, want_lse = da.linear_xent_forward(x, w, y)
    x2 = x.clone()
    x2[3, 5] = float("nan")
    x2[7] = float("inf")
    loss, lse = da.linear_xent_forward(x2, w, y)
    assert bool(torch.isnan(loss[3])) and not bool(torch.isfinite(loss[7]))
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[3] = keep[7] = False
    assert torch.equal(loss[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    dx, _ = da.linear_xent_backward(x2, w, y, lse, dl)
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isfinite(dx[keep]).all())


def test_large_logits_do_not_overflow():
    x, w, y, dl = _inputs(64, 300, 64, seed=12)
    x = (x.float() * 200).bfloat16()
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dw).all())
    loss64, lse64 = ref.xent(x, w, y, IGN)
    tol = (64 * 2.0 ** -23 + 2.0 ** -20) * (x.double().abs() @ w.double().abs().t()).amax(1) * 2 + 2.0 ** -14
    assert bool(((loss.double() - loss64).abs() <= 2 * tol).all())


def test_target_out_of_range_is_reported():
    x, w, y, dl = _inputs(140, 300, 64, seed=13, ignored=0.0)
    want, lse = da.linear_xent_forward(x, w, y)
    for bad in (300, -1, 2 ** 40):
        y2 = y.clone()
        y2[77] = bad
        with pytest.raises(da.DashError, match="a target") as e:
            da.linear_xent_forward(x, w, y2)
        assert e.value.status == da.DASH_ERR_BOUNDS
        loss, lse2 = da.linear_xent_forward(x, w, y2, check=False)
        assert bool(torch.isnan(loss[77])) and torch.equal(lse, lse2)
        ws = da.new_linear_xent_workspace(140, 300, 64, "cuda")
        dx, dw = da.linear_xent_backward(x, w, y2, lse, dl, workspace=ws, check=False)
        assert da.dash_attn_get_status(ws) == da.DASH_ERR_BOUNDS
        y3 = y.clone()
        y3[77] = IGN
        for a, b in zip((dx, dw), da.linear_xent_backward(x, w, y3, lse, dl)):
            assert torch.equal(a, b)


def test_bitwise_reproducible():
    x, w, y, dl = _inputs(700, 9001, 256, seed=14)
    ws = da.new_linear_xent_workspace(700, 9001, 256, "cuda")
    loss, lse = da.linear_xent_forward(x, w, y, workspace=ws)
    want = (loss, lse) + da.linear_xent_backward(x, w, y, lse, dl, workspace=ws)
    for _ in range(10):
        ws.random_(0, 255)
        loss, lse = da.linear_xent_forward(x, w, y, workspace=ws)
        got = (loss, lse) + da.linear_xent_backward(x, w, y, lse, dl, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_on_another_stream_and_in_a_graph():
    x, w, y, dl = _inputs(200, 1000, 128, seed=15)
    loss, lse = da.linear_xent_forward(x, w, y)
    want = (loss, lse) + da.linear_xent_backward(x, w, y, lse, dl)
    ws = da.new_linear_xent_workspace(200, 1000, 128, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, b = da.linear_xent_forward(x, w, y, workspace=ws, check=False)
        got = (a, b) + da.linear_xent_backward(x, w, y, b, dl, workspace=ws, check=False)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = da.linear_xent_forward(x, w, y, workspace=ws, check=False)
        got = (a, b) + da.linear_xent_backward(x, w, y, b, dl, workspace=ws, check=False)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_gradient_matches_differences_of_the_forward():
    """Along a direction: (L(x + h d) - L(x - h d)) / 2h against <dX, d>, with h d a whole
    number of bf16 steps so that both points are exact."""
    T, V, D = 64, 500, 64
    x, w, y, dl = _inputs(T, V, D, seed=16)
    x = x.float().clamp(-1.9, 1.9).mul(64).round().div(64).bfloat16()     # multiples of 2^-6
    d = torch.randint(0, 2, (T, D), device="cuda").mul(2).sub(1).float()
    h = 2.0 ** -6
    up, dn = (x.float() + h * d).bfloat16(), (x.float() - h * d).bfloat16()
    assert torch.equal(up.float() - dn.float(), 2 * h * d)
    L = lambda a: float((da.linear_xent_forward(a, w, y)[0].double() * dl.double()).sum())
    _, lse = da.linear_xent_forward(x, w, y)
    dx, _ = da.linear_xent_backward(x, w, y, lse, dl)
    got = float((dx.double() * d.double()).sum())
    # third-order term of the central difference: h^2 / 6 times the third derivative along d,
    # at most |dz|^3 per row with |dz| <= sum_i |w_i|; fp32 losses 2^-20 / 2h; bf16 of dX
    dz = w.double().abs().sum(1).max()
    tol = float((dl.double().abs() * (h * h / 6 * dz ** 3 + 2.0 ** -16 / h)).sum()
                + 2 * U * ref.xent_grad(x, w, y, dl, IGN)[2].abs().sum() * dz)
    assert abs((L(up) - L(dn)) / (2 * h) - got) <= tol


def test_waits_that_run_out_are_reported_and_the_context_survives():
    """The testing hook withholds the tiles: every wait for them runs out, the workspace says
    so, and the next call computes the normal result."""
    x, w, y, dl = _inputs(300, 600, 64, seed=17)
    ws = da.new_linear_xent_workspace(300, 600, 64, "cuda")
    loss, lse = da.linear_xent_forward(x, w, y, workspace=ws)
    want = (loss, lse) + da.linear_xent_backward(x, w, y, lse, dl, workspace=ws)
    try:
        da.dash_debug_set_sync(50_000_000, 1)
        da.linear_xent_forward(x, w, y, workspace=ws, check=False)
        assert da.dash_attn_get_status(ws) == da.DASH_ERR_SYNC_TIMEOUT
        da.linear_xent_backward(x, w, y, lse, dl, workspace=ws, check=False)
        assert da.dash_attn_get_status(ws) == da.DASH_ERR_SYNC_TIMEOUT
    finally:
        da.dash_debug_set_sync(0, 0)
    loss, lse = da.linear_xent_forward(x, w, y, workspace=ws)
    got = (loss, lse) + da.linear_xent_backward(x, w, y, lse, dl, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T,V,D", [(300, 900, 136), (700, 5003, 64), (2500, 700, 320)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_an_fp32_gradient_is_not_held_to_16_bits(T, V, D, accumulate):
    """dw in fp32 of more than 128 tokens: G enters it as two terms (u^2 |G|), so what is left
    beside the logits' error is the fp32 sums. They lie below half a step of bf16 where the
    targets dominate."""
    x, w, y, dl = _inputs(T, V, D, seed=T + 1)
    _, lse = da.linear_xent_forward(x, w, y)
    base = torch.randn(V, D, device="cuda").mul_(1e-3) if accumulate else None
    dw = base.clone() if accumulate else torch.full((V, D), float("nan"), device="cuda")
    da.linear_xent_backward(x, w, y, lse, dl, dw=dw, accumulate=accumulate)
    _, lse64 = ref.xent(x, w, y, IGN)
    _, dw64, G, gp = ref.xent_grad(x, w, y, dl, IGN)
    if accumulate:
        dw64 = dw64 + base.double()
    xd = x.double().abs()
    ez = (D * 2.0 ** -23 + 2.0 ** -22) * (xd @ w.double().abs().t()).amax(1)
    tol = 2 * ez + 2.0 ** -21 + 2.0 ** -14 + 2.0 ** -23 * lse64.abs()
    eG = U * U * G.abs() + gp * (tol[:, None] + ez[:, None] + 2.0 ** -20)
    bw = eG.t() @ xd + T * 2.0 ** -23 * (G.abs().t() @ xd) + 2.0 ** -24 * dw64.abs() * 1.01 + 1e-30
    assert bool(((dw.double() - dw64).abs() <= bw).all()), float(((dw.double() - dw64).abs() / bw).max())


@pytest.mark.parametrize("accumulate", [False, True])
def test_a_long_sum_of_one_sign_is_not_truncated(accumulate):
    """dw over 2^18 tokens whose terms have one sign. The tensor core truncates its additions of
    16 tokens, one or two steps of 2^-23 each; left to itself over 2^14 of them that is some
    3e-4. The bound is what segments of 1024 tokens, added to nearest, would leave at most: 64
    2^-22 within a segment and 2^8 2^-24 over them. With w = 0 the logits are 0 and p = 1/2 exactly; G is two terms (2^-16)."""
    T, V, D = 1 << 18, 2, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (1 + torch.rand(T, D, generator=g, device="cuda")).bfloat16()
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    dl = 0.5 + torch.rand(T, generator=g, device="cuda")
    base = torch.ones(V, D, device="cuda")
    _, lse = da.linear_xent_forward(x, w, y)
    dw = base.clone()
    da.linear_xent_backward(x, w, y, lse, dl, dw=dw, accumulate=accumulate)
    want = 0.5 * (dl.double()[:, None] * x.double()).sum(0)
    want = torch.stack((-want, want)) + (base.double() if accumulate else 0)
    assert bool(((dw.double() - want).abs() <= (64 * 2.0 ** -22 + 2.0 ** -16 + 2.0 ** -16) * want.abs()).all())


def test_a_long_sum_into_bf16_with_and_without_the_tile_store():
    """More than 16384 tokens in one call, whose products reach dw in several segments."""
    T, V, D = 33001, 600, 72
    x, w, y, dl = _inputs(T, V, D, seed=21)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)
    base = torch.randn(V, D, device="cuda").mul_(1e-3).bfloat16()
    dw = base.clone()
    da.linear_xent_backward(x, w, y, lse, dl, dw=dw, accumulate=True)
    _check(x, w, y, dl, loss, lse, dx, dw, base=base)


@pytest.mark.parametrize("T,V,D", [(20, 700, 1032), (64, 300, 1096), (130, 520, 3080), (64, 300, 4096)])
def test_hidden_sizes_of_several_segments(T, V, D):
    """K of the logits in one and more segments of 1024, the last of them short."""
    x, w, y, dl = _inputs(T, V, D, seed=D)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


def test_a_long_logit_of_one_sign_is_not_truncated():
    """Logits over K = 16384 whose products have one sign: 64 additions of 16 products within a
    segment of 1024, one or two steps of 2^-23 of the segment's growing sum each (32 2^-22 at
    most), 15 additions of segments and the scalings to nearest. One sum over all of K would be
    2e-5 too small, more than twice this bound."""
    T, V, D = 64, 300, 16384
    g = torch.Generator(device="cuda").manual_seed(22)
    x = (0.5 + torch.rand(T, D, generator=g, device="cuda")).bfloat16()
    w = ((0.5 + torch.rand(V, D, generator=g, device="cuda")) * (60.0 / D)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    loss, lse = da.linear_xent_forward(x, w, y)
    loss64, lse64 = ref.xent(x, w, y, IGN)
    tol = (32 * 2.0 ** -22 + 20 * 2.0 ** -24) * lse64.abs() + 2.0 ** -19
    assert bool(((lse.double() - lse64).abs() <= tol).all())
    assert bool(((loss.double() - loss64).abs() <= 2 * tol).all())


def test_pieces_whose_products_are_not_split():
    """dX summed over the pieces of the vocabulary tile by tile: the first piece, one in the
    middle and the last, with more tiles than a split of K starts from."""
    T, V, D = 4096, 66000, 520
    x, w, y, dl = _inputs(T, V, D, seed=23)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


def test_a_long_range_of_the_vocabulary_in_one_unit():
    """dX over 30000 ids in one unit of work: several segments of K."""
    T, V, D = 2500, 30000, 1024
    x, w, y, dl = _inputs(T, V, D, seed=24)
    loss, lse = da.linear_xent_forward(x, w, y)
    dx, dw = da.linear_xent_backward(x, w, y, lse, dl)
    _check(x, w, y, dl, loss, lse, dx, dw)


@pytest.mark.parametrize("dwt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,D", [(64, 999, 200), (64, 524300, 8), (4096, 40000, 64), (1300, 20000, 2048)])
def test_accumulation_by_terms_pieces_and_launches(T, V, D, dwt):
    """dw added to what it holds: two terms of G in the empty half of a tile, those over two
    pieces, several pieces of many tokens, and products in launches of their own."""
    x, w, y, dl = _inputs(T, V, D, seed=T + D)
    loss, lse = da.linear_xent_forward(x, w, y)
    base = torch.randn(V, D, device="cuda").mul_(1e-3).to(dwt)
    dw = base.clone()
    dx, _ = da.linear_xent_backward(x, w, y, lse, dl, dw=dw, accumulate=True)
    _check(x, w, y, dl, loss, lse, dx, dw, base=base)
