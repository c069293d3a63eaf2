"""CPU: workspaces of cross attention for batches that may be empty and for long states, and where its
gradients may lie."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built
from tests.test_train_devices import library, on1  # noqa: F401


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def test_a_workspace_for_no_batch_is_one_for_one():
    for forward_only in (False, True):
        ws = [da.new_cross_attn_workspace(B, 4, 2000, 4, 2, 64, "cpu", forward_only) for B in (0, 1)]
        assert ws[0].numel() == ws[1].numel() >= 256
    with pytest.raises(da.DashError):
        da.new_cross_attn_workspace(0, 4, 2000, 4, 2, 60, "cpu")


def test_workspaces_of_long_states():
    """A key range takes at most 65536 keys, so longer states leave partials of every row, fp32, whatever
    the number of rows; up to that length many rows leave none."""
    rows = 77 * 256
    one, two, many = (da.dash_cross_attn_fwd_workspace_size(1, rows, Sk, 1, 1, 64) for Sk in (65536, 65537, 1 << 22))
    assert one == 256
    assert rows * 2 * 65 * 4 <= two <= rows * 2 * 65 * 4 + 1024
    assert rows * 64 * 65 * 4 <= many <= rows * 64 * 65 * 4 + 1024
    one, many = (da.dash_cross_attn_bwd_workspace_size(1, rows, Sk, 1, 1, 64) for Sk in (65536, 1 << 22))
    assert many >= one and many >= 256 + rows * (8 + 64 * 64 * 4)


def test_gradients_lie_over_nothing_else(library):  # noqa: F811
    q, k, v = (on1(torch.zeros(1, 128, H, 16, dtype=torch.bfloat16)) for H in (2, 1, 1))
    o, do, lse = on1(torch.zeros_like(q)), on1(torch.zeros_like(q)), on1(torch.zeros(1, 2, 128))
    both = on1(torch.zeros_like(k))
    for kw in (dict(dq=q), dict(dk=k), dict(dv=v), dict(dv=k), dict(dq=do), dict(dq=o), dict(dk=both, dv=both)):
        with pytest.raises(ValueError, match="lies over"):
            da.cross_attn_backward(q, k, v, o, do, lse, 1.0, **kw)
    fused = on1(torch.zeros(1, 128, 4, 16, dtype=torch.bfloat16))
    got = da.cross_attn_backward(q, k, v, o, do, lse, 1.0, dq=fused[:, :, :2], dk=fused[:, :, 2:3], dv=fused[:, :, 3:])
    assert got[0].data_ptr() == fused.data_ptr() and got[2].shape == v.shape
