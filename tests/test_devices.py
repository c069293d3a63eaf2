"""CPU: the attention's and the split-K product's calls, and the status read, run on their
tensors' device whichever device is current (the library and the devices are stood in for)."""
import contextlib

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from reproducible_deterministic_attn_gb300 import dash_attn as core
from tests.test_train_devices import Library, on1


@pytest.fixture
def library(monkeypatch):
    state = {"current": 0}

    @contextlib.contextmanager
    def device_of(t):
        was, state["current"] = state["current"], t.get_device()
        try:
            yield
        finally:
            state["current"] = was

    lib = Library(state)
    empty = torch.empty
    monkeypatch.setattr(core, "load", lambda: lib)
    monkeypatch.setattr(core, "_stream", lambda t, stream: 0)
    monkeypatch.setattr(torch.cuda, "device_of", device_of)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: on1(empty(*a, **k)))
    return lib


def _qkv(n):
    return [on1(torch.zeros(1, 128, 1, 64, dtype=torch.bfloat16)) for _ in range(n)]


LSE = torch.zeros(1, 1, 128)
CALLS = {
    "dash_attn_fwd": lambda: da.attn_forward(*_qkv(3), 0.125, True),
    "dash_attn_fwd_ex": lambda: core.dash_attn_fwd_ex(*_qkv(4), on1(LSE), 0.125, 1),
    "dash_attn_bwd": lambda: da.attn_backward(*_qkv(5), on1(LSE), 0.125, True),
    "dash_attn_bwd_static": lambda: core.dash_attn_bwd_static(*_qkv(5), on1(LSE), *_qkv(3), 0.125, 1, 0, 1),
    "dash_gemm_splitk": lambda: da.gemm_splitk(on1(torch.zeros(128, 64)), on1(torch.zeros(128, 64)), 2),
    "dash_attn_get_status": lambda: da.dash_attn_get_status(on1(torch.zeros(64, dtype=torch.uint8))),
}


@pytest.mark.parametrize("name", CALLS)
def test_runs_on_the_tensors_device(library, name):
    CALLS[name]()
    assert name in [n for n, _ in library.calls]
    assert all(dev == 1 for n, dev in library.calls if not n.endswith("_size")), library.calls
    assert library.state["current"] == 0
