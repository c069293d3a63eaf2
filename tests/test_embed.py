"""GPU: embedding lookup and its gradient against the float64 definition.

Tolerances: the lookup is one multiplication (fp32, rounded once) and the rounding of its
result, u = eps / 2 of the type, at most u (1 + 2^-15) relative for 16-bit types, 2^-23 for
fp32 (the multiplication by a float32 scale); below the normal range half the smallest
number. The gradient sums c rows in fp32 (c 2^-24 of the sum of absolute values; twice that
for the joins), times scale, rounded once."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

TYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _half_step(t):
    return torch.finfo(t).eps / 2


def _grad_ok(got, want, absum, count, t, scale, base=None):
    tol = 2 * (count + 1) * 2.0 ** -24 * abs(scale) * absum
    if base is not None:
        want = want + base.double()
    tol = tol + (_half_step(t) + 2.0 ** -23) * (want.abs() + tol) + TINY[t]
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def _run_grad(T, V, D, ids, t, out_t=None, scale=0.75, padding_idx=None, accumulate=False, seed=1, strided=False):
    g = _gen(seed)
    dout = torch.randn(T, D + (24 if strided else 0), generator=g, device="cuda").to(t)[:, :D]
    base = torch.randn(V, D, generator=g, device="cuda").to(out_t or t) if accumulate else None
    if accumulate:
        out = base.clone()
    else:
        out = torch.full((V, D), float("nan"), dtype=out_t or t, device="cuda")
    got = da.embed_backward(dout, ids, V, scale, padding_idx=padding_idx, dtable=out, accumulate=accumulate)
    assert got is out
    want = ref.embed_grad(dout, ids.long(), V, scale, padding_idx)
    absum = ref.embed_grad(dout.abs(), ids.long(), V, 1.0, padding_idx)
    count = torch.bincount(ids.long(), minlength=V).double()[:, None]
    _grad_ok(got, want, absum, count, out_t or t, scale, base)
    if not accumulate:
        absent = count[:, 0] == 0
        assert bool((got[absent] == 0).all())
    else:
        assert torch.equal(got[count[:, 0] == 0], base[count[:, 0] == 0])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (3, 7, 5), (33, 100, 64), (257, 50, 1000), (64, 300, 1023), (5, 9, 4104)])
def test_lookup(t, T, V, D):
    g = _gen(T + D)
    table = torch.randn(V, D, generator=g, device="cuda").to(t)
    for idt in (torch.int32, torch.int64):
        ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(idt)
        assert torch.equal(da.embed_forward(table, ids), table[ids.long()])
        got = da.embed_forward(table, ids, 1.7)
        want = ref.embed(table, ids.long(), 1.7)
        u = _half_step(t) * (1 + 2.0 ** -15) + 2.0 ** -23
        assert bool(((got.double() - want).abs() <= u * want.abs() + TINY[t]).all())


def test_lookup_shapes_strides_and_no_tokens():
    table = torch.randn(50, 88, device="cuda").bfloat16()
    wide = torch.zeros(50, 120, device="cuda", dtype=torch.bfloat16)[:, 3:91]
    wide.copy_(table)
    ids = torch.randint(0, 50, (4, 6), device="cuda")
    assert torch.equal(da.embed_forward(table, ids), table[ids])
    assert torch.equal(da.embed_forward(wide, ids), table[ids])
    assert da.embed_forward(table, ids[:0]).shape == (0, 6, 88)


def test_lookup_into_strided_rows():
    """The C call's output stride: the elements between the rows stay as they are."""
    for D, ld in ((64, 72), (64, 67), (33, 40)):
        table = torch.randn(20, D, device="cuda").bfloat16()
        ids = torch.randint(0, 20, (9,), device="cuda")
        out = torch.full((9, ld), 5.0, dtype=torch.bfloat16, device="cuda")
        assert da.load().dash_embed_fwd(table.data_ptr(), ids.data_ptr(), out.data_ptr(), None, 9, 20, D, D, ld, 1.0,
                                        da.DASH_BF16, 64, torch.cuda.current_stream().cuda_stream) == da.DASH_OK
        assert torch.equal(out[:, :D], table[ids]) and bool((out[:, D:] == 5).all())


def test_lookup_out_of_range_gives_nan_rows_and_the_status():
    table = torch.randn(50, 64, device="cuda").bfloat16()
    ids = torch.tensor([3, 50, -1, 7, 2 ** 40], device="cuda")
    status = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    out = da.embed_forward(table, ids, 2.0, status=status)
    assert int(status) == da.DASH_ERR_BOUNDS
    assert bool(torch.isnan(out[[1, 2, 4]]).all()) and torch.equal(out[[0, 3]], table[[3, 7]] * 2)
    da.embed_forward(table, ids[:1], status=status)
    assert int(status) == da.DASH_OK


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (2, 1, 8), (31, 3, 40), (32, 2, 64), (33, 2, 64), (65, 600, 33),
                                   (1000, 70, 129), (4097, 700, 256), (3000, 300000, 16), (20000, 5, 24)])
def test_gradient(t, T, V, D):
    ids = torch.randint(0, V, (T,), generator=_gen(T), device="cuda")
    _run_grad(T, V, D, ids, t)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_gradient_into_fp32_and_accumulated(t):
    ids = torch.randint(0, 90, (700,), generator=_gen(2), device="cuda").to(torch.int32)
    _run_grad(700, 200, 72, ids, t, torch.float32)
    _run_grad(700, 200, 72, ids, t, torch.float32, accumulate=True)
    _run_grad(700, 200, 72, ids, t, t, accumulate=True)
    _run_grad(700, 200, 71, ids, t, t, accumulate=True)
    _run_grad(700, 200, 72, ids, t, strided=True)


def test_gradient_of_one_hot_id_and_skewed_ids():
    for T in (32, 64, 1024, 4100):
        _run_grad(T, 10, 136, torch.full((T,), 4, device="cuda"), torch.bfloat16)
    u = torch.rand(9000, generator=_gen(3), device="cuda")
    _run_grad(9000, 4000, 64, (u ** 6 * 4000).long().clamp_(0, 3999), torch.bfloat16)


def test_padding_ids_are_left_out():
    ids = torch.randint(0, 8, (500,), generator=_gen(4), device="cuda")
    _run_grad(500, 8, 64, ids, torch.float32, padding_idx=3)
    dout = torch.randn(500, 64, device="cuda")
    got = da.embed_backward(dout, ids, 8, padding_idx=3)
    assert float(got[3].abs().max()) == 0
    got = da.embed_backward(dout, torch.full_like(ids, 3), 8, padding_idx=3)
    assert float(got.abs().max()) == 0


def test_no_tokens_gives_zeros():
    out = torch.full((40, 16), float("nan"), device="cuda")
    da.embed_backward(torch.empty(0, 16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 40, dtable=out)
    assert float(out.abs().max()) == 0


def test_gradient_id_out_of_range_contributes_nothing_and_is_reported():
    ids = torch.randint(0, 30, (400,), generator=_gen(5), device="cuda")
    dout = torch.randn(400, 64, device="cuda").bfloat16()
    bad = ids.clone()
    bad[100] = 30
    bad[101] = -7
    with pytest.raises(da.DashError, match="a token id"):
        da.embed_backward(dout, bad, 30)
    ws = da.new_embed_workspace(400, 30, 64, "cuda")
    got = da.embed_backward(dout, bad, 30, workspace=ws, check=False)
    assert da.dash_attn_get_status(ws) == da.DASH_ERR_BOUNDS
    keep = (bad >= 0) & (bad < 30)
    _grad_ok(got, ref.embed_grad(dout[keep], bad[keep], 30, 1.0),
             ref.embed_grad(dout[keep].abs(), bad[keep], 30, 1.0), 40, torch.bfloat16, 1.0)


def test_nan_and_inf_stay_in_their_ids():
    ids = torch.tensor([0, 1, 2, 1, 0], device="cuda")
    dout = torch.ones(5, 32, device="cuda")
    dout[1] = float("inf")
    dout[2] = float("nan")
    got = da.embed_backward(dout, ids, 4)
    assert bool((got[0] == 2).all()) and bool(torch.isinf(got[1]).all()) and bool(torch.isnan(got[2]).all())
    assert bool((got[3] == 0).all())


def test_bitwise_reproducible_on_streams_and_in_a_graph():
    ids = (torch.rand(6000, generator=_gen(6), device="cuda") ** 4 * 900).long()
    dout = torch.randn(6000, 200, generator=_gen(7), device="cuda").bfloat16()
    ws = da.new_embed_workspace(6000, 900, 200, "cuda")
    want = da.embed_backward(dout, ids, 900, workspace=ws)
    for _ in range(10):
        ws.random_(0, 255)
        assert torch.equal(da.embed_backward(dout, ids, 900, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = da.embed_backward(dout, ids, 900, workspace=ws, check=False)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = da.embed_backward(dout, ids, 900, workspace=ws, check=False)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_rows_beyond_32_bit_offsets():
    """A table of more than 2^31 elements: its last rows are read and written."""
    V, D = (1 << 20) + 3, 2056
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[V - 1] = torch.arange(D, device="cuda").bfloat16()
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    out = da.embed_forward(table, ids)
    assert torch.equal(out[0], table[V - 1]) and float(out[1].abs().max()) == 0
    grad = da.embed_backward(out, ids, V, dtable=table)
    assert torch.equal(grad[V - 1].float(), (2 * out[0].float()).bfloat16().float())
    assert float(grad[:V - 1].abs().max()) == 0


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,D", [(32769, 5, 24), (40000, 70, 129), (70001, 300000, 16)])
def test_gradient_of_more_tokens_than_a_warp_holds(t, T, V, D):
    """Above 32768 tokens a warp of the sort has more strips than it keeps and reads them twice."""
    ids = torch.randint(0, V, (T,), generator=_gen(T), device="cuda")
    _run_grad(T, V, D, ids, t)
    _run_grad(T, V, D, ids.to(torch.int32), t, torch.float32, padding_idx=3, accumulate=True)
