"""CPU: workspaces of cross attention for batches that may be empty."""
import pytest

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built


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
