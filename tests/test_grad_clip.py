"""GPU: gradient norm and clipping against the float64 definition.

Tolerances: squares are summed in fp32 by a thread over at most 64 elements of a piece plus a
tree of 4 (68 2^-24 relative, all terms positive), then in fp64; the root halves that, the
norm's own rounding adds 2^-24: 2^-18 covers it. A clipped value: the factor's rounding and
error (2^-18 + 2^-24), one product, its rounding u = eps / 2."""
import math

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from oracle import train_ops as ref
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

TYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
NORM_REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _tensors(sizes, types, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def _check(grads, got, norm, max_norm):
    n64, want = ref.clip(grads, max_norm)
    assert abs(float(norm) - float(n64)) <= NORM_REL * float(n64)
    for g, o, w in zip(grads, got, want):
        if float(n64) <= max_norm:
            assert torch.equal(g, o)
        elif o.numel():
            u = torch.finfo(o.dtype).eps / 2
            err = (o.double() - w).abs()
            assert bool((err <= (u + 2.0 ** -17) * w.abs() + TINY[o.dtype]).all())


@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES])
@pytest.mark.parametrize("sizes", [[1], [7, 1, 3], [32768, 32769, 32767, 0, 5], [100003, 8, 1 << 20, 17]])
@pytest.mark.parametrize("factor", [0.3, 2.0])
def test_in_place_and_into_buffers(types, sizes, factor):
    grads = _tensors(sizes, types, seed=len(sizes))
    keep = [g.clone() for g in grads]
    max_norm = factor * float(ref.clip(grads, math.inf)[0])
    outs = [torch.full_like(g, float("nan")) for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads, outs), max_norm)
    _check(keep, got, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    plan = da.grad_clip_plan(grads)
    norm2, got2 = da.grad_clip(plan, max_norm)
    assert torch.equal(norm, norm2)
    for a, b in zip(outs, got2):
        assert torch.equal(a, b)


def test_unaligned_tensors():
    buf = torch.randn(70001, device="cuda").bfloat16()
    for lo in (1, 2, 3, 5):
        grads = [buf[lo:].clone()[0:0], buf[lo:]]
        keep = [g.clone() for g in grads]
        out = [torch.empty_like(g) for g in grads]
        norm, got = da.grad_clip(da.grad_clip_plan(grads, out), 1.0)
        _check(keep, got, norm, 1.0)


def test_many_tensors():
    grads = _tensors([1 + (i * 37) % 4000 for i in range(1500)], TYPES, seed=3)
    keep = [g.clone() for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads), 2.0)
    _check(keep, got, norm, 2.0)


def test_zeros_and_limits():
    grads = _tensors([5000, 70000], [torch.float32], std=0.0)
    norm, got = da.grad_clip(da.grad_clip_plan(grads), 1.0)
    assert float(norm) == 0 and all(float(g.abs().max()) == 0 for g in got)
    grads = _tensors([100], [torch.float32], seed=4)
    keep = grads[0].clone()
    norm, got = da.grad_clip(da.grad_clip_plan(grads), math.inf)
    assert torch.equal(got[0], keep)
    norm, got = da.grad_clip(da.grad_clip_plan(grads), 0.0)
    assert float(got[0].abs().max()) == 0


@pytest.mark.parametrize("t,scale", [(torch.float32, 2.0 ** 100), (torch.float32, 2.0 ** -100),
                                     (torch.float32, 2.0 ** -140), (torch.bfloat16, 2.0 ** 90),
                                     (torch.bfloat16, 2.0 ** -90), (torch.float16, 2.0 ** -20)])
def test_squares_beyond_the_range_of_fp32(t, scale):
    """The squares leave fp32's range, the norm does not; other tensors are of the usual size
    or zero, and one thread's elements mix both."""
    g = (torch.randn(50021, device="cuda", dtype=torch.float64) * scale).to(t)
    keep = g.clone()
    n64 = float(ref.clip([g], math.inf)[0])
    norm, got = da.grad_clip(da.grad_clip_plan([g]), math.inf)
    assert abs(float(norm) - n64) <= NORM_REL * n64 + 2.0 ** -149
    norm, got = da.grad_clip(da.grad_clip_plan([g, torch.zeros(4000, device="cuda")]), n64 / 2)
    w = keep.double() * 0.5
    u = torch.finfo(t).eps / 2
    assert bool(((got[0].double() - w).abs() <= (u + 2.0 ** -17) * w.abs() + TINY[t]).all())
    if scale > 1:
        mixed = torch.randn(40000, device="cuda")
        mixed[::7] *= scale
        n64 = float(ref.clip([mixed], math.inf)[0])
        norm, _ = da.grad_clip(da.grad_clip_plan([mixed]), math.inf)
        assert abs(float(norm) - n64) <= NORM_REL * n64


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    grads = _tensors([40000, 300], [torch.bfloat16, torch.float32], seed=5)
    grads[0][31234] = bad
    keep = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads, outs), 1.0)
    assert not math.isfinite(float(norm)) and (math.isnan(float(norm)) == math.isnan(bad))
    same = lambda a, b: torch.equal(a.nan_to_num(nan=123.0), b.nan_to_num(nan=123.0))
    assert all(same(a, b) for a, b in zip(got, keep))
    da.grad_clip(da.grad_clip_plan(grads), 1.0)
    assert all(same(a, b) for a, b in zip(grads, keep))


def test_bitwise_reproducible_streams_and_graph():
    grads = _tensors([3000017, 70001, 9, 1 << 19], TYPES, seed=6)
    outs = [torch.empty_like(g) for g in grads]
    plan = da.grad_clip_plan(grads, outs)
    norm, got = da.grad_clip(plan, 3.0)
    want = [norm.clone()] + [t.clone() for t in got]
    for _ in range(10):
        norm, got = da.grad_clip(plan, 3.0)
        assert all(torch.equal(a, b) for a, b in zip(want, [norm] + got))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        da.grad_clip(plan, 3.0)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm, got = da.grad_clip(plan, 3.0)
    for t in got:
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [norm] + got))


def test_something_else_than_a_plan_gives_nan_and_touches_nothing():
    grads = _tensors([100000, 500], [torch.float32], seed=7)
    keep = [g.clone() for g in grads]
    plan = da.grad_clip_plan(grads)
    lib, norm = da.load(), torch.zeros((), device="cuda")
    blank = torch.zeros(plan.table.numel(), dtype=torch.uint8, device="cuda")
    for table, size in ((blank, blank.numel()), (plan.table, plan.table.numel() - 24 * 20)):
        norm.zero_()
        assert lib.dash_grad_clip(table.data_ptr(), size, 0.5, norm.data_ptr(), 0) == da.DASH_OK
        torch.cuda.synchronize()
        assert math.isnan(float(norm)) and all(torch.equal(a, b) for a, b in zip(grads, keep))
    got, _ = da.grad_clip(plan, 0.5)
    assert math.isfinite(float(got))


@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES])
@pytest.mark.parametrize("factor", [0.3, 2.0])
def test_lists_whose_pieces_are_whole(types, factor):
    """More than 20 million elements, so that pieces have 32768 and a thread its full number of
    loads in flight, aligned and not; into buffers and in place."""
    buf = _tensors([9000002], [types[0]], seed=8)[0]
    grads = _tensors([16777221, 70001, 33], types, seed=9) + [buf[1:]]
    keep = [g.clone() for g in grads]
    max_norm = factor * float(ref.clip(grads, math.inf)[0])
    outs = [torch.full_like(g, float("nan")) for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads, outs), max_norm)
    _check(keep, got, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    norm2, got2 = da.grad_clip(da.grad_clip_plan(grads), max_norm)
    assert torch.equal(norm, norm2)
    assert all(torch.equal(a, b) for a, b in zip(outs, got2))


@pytest.mark.parametrize("short", [1, 30])
def test_a_plan_of_more_pieces_than_blocks_in_a_buffer_too_short(short):
    """The whole table is there, but the call says that its buffer ends some entries earlier."""
    grads = _tensors([700 * 4096], [torch.float32], seed=11)
    keep = [g.clone() for g in grads]
    plan = da.grad_clip_plan(grads)
    lib, norm = da.load(), torch.zeros((), device="cuda")
    size = plan.table.numel() - 256 - 24 * short
    assert lib.dash_grad_clip(plan.table.data_ptr(), size, 0.5, norm.data_ptr(), 0) == da.DASH_OK
    torch.cuda.synchronize()
    assert math.isnan(float(norm)) and all(torch.equal(a, b) for a, b in zip(grads, keep))
    got, _ = da.grad_clip(plan, 0.5)
    assert math.isfinite(float(got))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_a_norm_beyond_fp32_leaves_the_values(t):
    """The elements are finite and so is their norm in 64 bits; in 32, as the caller gets it, it
    is not."""
    grads = [torch.full((3,), 3e38, dtype=t, device="cuda"), torch.randn(5000, device="cuda")]
    keep = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads, outs), 1.0)
    assert float(norm) == math.inf and all(torch.equal(a, b) for a, b in zip(got, keep))
    norm, _ = da.grad_clip(da.grad_clip_plan(grads), 1.0)
    assert float(norm) == math.inf and all(torch.equal(a, b) for a, b in zip(grads, keep))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,max_norm", [(1e36, 1e-6), (1e33, 1e-9), (1e36, 1e-37), (1.0, 1e-38)])
def test_a_limit_far_below_the_norm(t, size, max_norm):
    """The factor is below fp32's normal range, or the clipped values are."""
    grads = [(torch.randn(50021, device="cuda", dtype=torch.float64) * size).to(t),
             torch.randn(300, device="cuda")]
    keep = [g.clone() for g in grads]
    outs = [torch.full_like(g, float("nan")) for g in grads]
    norm, got = da.grad_clip(da.grad_clip_plan(grads, outs), max_norm)
    _check(keep, got, norm, max_norm)
    norm, got = da.grad_clip(da.grad_clip_plan(grads), max_norm)
    assert all(torch.equal(a, b) for a, b in zip(outs, got))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("aligned", [True, False])
def test_mostly_zero_rows_and_single_values_among_zeros(t, aligned):
    """A table's gradient whose rows are mostly zero, of either sign, and threads that hold one
    value, small enough that its square is lost in fp32, among zeros."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(3001, 1024, generator=g, device="cuda").to(t)
    x[torch.rand(3001, generator=g, device="cuda") < 0.8] = -0.0
    low = torch.zeros(200000, device="cuda", dtype=t)
    low[:3001] = -0.0
    low[::4099] = torch.finfo(t).tiny * 0.75
    x, low = (v.reshape(-1)[0 if aligned else 1:] for v in (x, low))
    for grads in ([x], [low], [x, low], [torch.full_like(x, -0.0)]):
        n64 = float(ref.clip(grads, math.inf)[0])
        norm, _ = da.grad_clip(da.grad_clip_plan(grads), math.inf)
        assert abs(float(norm) - n64) <= NORM_REL * n64 + 2.0 ** -149


def test_a_plan_dropped_while_another_stream_still_uses_it():
    """Its memory is not given out again before that stream's work has ended."""
    grads = _tensors([5000, 70001], [torch.float32], seed=13)
    want = [g.clone() for g in grads]
    want_norm = da.grad_clip(da.grad_clip_plan(want), 1.0)[0].clone()
    plan = da.grad_clip_plan(grads)
    where, size = plan.table.data_ptr(), plan.table.numel()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    norm, got = da.grad_clip(plan, 1.0, stream=s)
    del plan
    new = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != where for t in new)
    s.synchronize()
    assert torch.equal(norm, want_norm) and all(torch.equal(a, b) for a, b in zip(got, want))
