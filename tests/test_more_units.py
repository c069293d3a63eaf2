"""GPU: cross attention where a CTA has many tasks, units of unlike lengths and units without keys, against
the float64 definition; group norm and rotation over several axes of tensors whose parts lie 2^32
elements apart, against the same values side by side (the same sums in the same order: equal bits)."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built, has_gpu
from tests.test_cross_attn import _check_backward, _check_forward, _inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

FAR = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D,lens", [
    (3, 1311, 700, 20, 5, 128, (700, 0, 131)),
    (2, 2050, 385, 11, 11, 64, (257, 385)),
    (9, 700, 260, 24, 8, 80, (260, 1, 128, 129, 0, 256, 17, 200, 3)),
    (2, 3001, 128, 30, 6, 128, (128, 127)),
    (40, 130, 300, 6, 6, 128, None),
    (5, 1, 3000, 64, 4, 128, (3000, 2, 1025, 0, 2999)),
])
def test_many_tasks_and_units(B, Sq, Sk, Hq, Hk, D, lens):
    x = _inputs(B, Sq, Sk, Hq, Hk, D, lens, seed=31)
    ws = da.new_cross_attn_workspace(B, Sq, Sk, Hq, Hk, D, "cuda")
    first = None
    for _ in range(4):
        o, lse = da.cross_attn_forward(x["q"], x["k"], x["v"], x["scale"], x["t"], workspace=ws)
        got = (o, lse, *da.cross_attn_backward(x["q"], x["k"], x["v"], o, x["do"], lse, x["scale"], x["t"],
                                               workspace=ws))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    _check_forward(x, *first[:2])
    _check_backward(x, *first)


def _far(t, dim):
    """A copy of t whose parts along `dim` lie 2^32 elements apart."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    strides = list(t.contiguous().stride())
    strides[dim] = FAR
    flat = torch.empty(FAR * (t.shape[dim] - 1) + t.numel(), dtype=t.dtype, device="cuda")
    out = flat.as_strided(t.shape, strides)
    out.copy_(t)
    return out


@pytest.mark.parametrize("S,C,G", [(70, 96, 8), (30011, 64, 4), (41, 250, 25)])
def test_group_norm_of_samples_far_apart(S, C, G):
    x = torch.randn(2, S, C, device="cuda").bfloat16()
    dy, w, b = torch.randn_like(x), torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    far = _far(x, 0)
    want = da.group_norm_act_forward(x, w, b, G)
    got = da.group_norm_act_forward(far, w, b, G)
    want += da.group_norm_act_backward(dy, x, w, b, *want[1:], G)
    got += da.group_norm_act_backward(dy, far, w, b, *got[1:], G)
    assert all(torch.equal(a, c) for a, c in zip(want, got))


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("R,interleaved", [(64, False), (64, True), (24, False)])
def test_rotation_of_parts_far_apart(dim, R, interleaved):
    shape = [2, 9, 2, 64]
    shape[dim] = 2
    q, k = torch.randn(shape, device="cuda").bfloat16(), torch.randn(shape, device="cuda").bfloat16()
    sections = (R // 4, R // 8, R // 8)
    cos, sin = da.rope_axes_table(50, sections)
    pos = torch.randint(0, 50, (3, *shape[:2]), device="cuda")
    w = torch.rand(64, device="cuda") + 0.5
    far = _far(q, dim)
    at = (w, w, cos, sin, pos, sections)
    want = da.qk_norm_rope_axes_forward(q, k, *at, interleaved=interleaved)
    got = da.qk_norm_rope_axes_forward(far, k, *at, interleaved=interleaved)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    want += da.qk_norm_rope_axes_backward(dq, dk, q, k, *at, interleaved=interleaved)
    got += da.qk_norm_rope_axes_backward(dq, dk, far, k, *at, interleaved=interleaved, dq=_far(q, dim))
    assert all(torch.equal(a, c) for a, c in zip(want, got))
