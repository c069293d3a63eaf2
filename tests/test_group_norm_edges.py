"""GPU: group norm at the edges of what it accepts, against the float64 definition."""
import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
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
