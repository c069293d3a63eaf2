"""CPU: the training-step operators run on their tensors' device whichever device is current.
The library, the tensors' device index and torch's current device are stood in for."""
import contextlib

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from reproducible_deterministic_attn_gb300 import train_ops


class On1(torch.Tensor):
    """A host tensor that says it lies on cuda:1."""

    def get_device(self):
        return 1


def on1(t):
    return t.as_subclass(On1)


class Library:
    """Records the current device of every call; sizes are some bytes, statuses are OK."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.state["current"]))
            return 64 if name.endswith("_size") else 0
        return call


@pytest.fixture
def library(monkeypatch):
    state = {"current": 0}

    @contextlib.contextmanager
    def device(index):
        was, state["current"] = state["current"], index
        try:
            yield
        finally:
            state["current"] = was

    lib = Library(state)
    empty = torch.empty
    monkeypatch.setattr(train_ops._core, "load", lambda: lib)
    monkeypatch.setattr(train_ops, "_current_device", lambda: state["current"], raising=False)
    monkeypatch.setattr(train_ops, "_stream", lambda dev: 0)
    monkeypatch.setattr(train_ops, "dash_attn_get_status",
                        lambda ws: lib.calls.append(("status", state["current"])) or 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: on1(empty(*a, **k)))
    return lib


def _qk():
    q, k = on1(torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)), on1(torch.zeros(1, 4, 1, 16, dtype=torch.bfloat16))
    w, c = on1(torch.ones(16)), on1(torch.zeros(8, 8))
    return q, k, w, w, c, c


def _xent():
    return (on1(torch.zeros(4, 16, dtype=torch.bfloat16)), on1(torch.zeros(9, 16, dtype=torch.bfloat16)),
            on1(torch.zeros(4, dtype=torch.int64)))


CALLS = {
    "dash_embed_fwd": lambda: da.embed_forward(on1(torch.zeros(9, 16)), on1(torch.zeros(4, dtype=torch.int64))),
    "dash_embed_bwd": lambda: da.embed_backward(on1(torch.zeros(4, 16)), on1(torch.zeros(4, dtype=torch.int64)), 9),
    "dash_qk_norm_rope_fwd": lambda: da.qk_norm_rope_forward(*_qk()),
    "dash_qk_norm_rope_bwd": lambda: da.qk_norm_rope_backward(*_qk()[:2], *_qk()),
    "dash_linear_xent_fwd": lambda: da.linear_xent_forward(*_xent()),
    "dash_linear_xent_bwd": lambda: da.linear_xent_backward(*_xent(), on1(torch.zeros(4)), on1(torch.zeros(4))),
    "dash_grad_clip_plan": lambda: da.grad_clip_plan([on1(torch.zeros(9))]),
    "dash_grad_clip": lambda: da.grad_clip(da.grad_clip_plan([on1(torch.zeros(9))]), 1.0),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_runs_on_the_tensors_device(library, name, current):
    library.state["current"] = current
    CALLS[name]()
    assert name in [n for n, _ in library.calls]
    assert all(dev == 1 for n, dev in library.calls if not n.endswith("_size")), library.calls
    assert library.state["current"] == current


def test_a_stream_of_another_device_is_refused(library):
    class Stream:
        device = torch.device("cuda", 0)

    real, torch.cuda.Stream = torch.cuda.Stream, Stream
    try:
        with pytest.raises(ValueError, match="stream: expected"):
            da.embed_forward(on1(torch.zeros(9, 16)), on1(torch.zeros(4, dtype=torch.int64)), stream=Stream())
    finally:
        torch.cuda.Stream = real
    assert not library.calls
