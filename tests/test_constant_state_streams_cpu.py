"""A stream of another device is refused before anything is allocated or launched."""
from types import SimpleNamespace

import pytest
import torch

import causal_prefix_scan_gb300 as hla
from causal_prefix_scan_gb300 import _build

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def calls():
    x, row, state = torch.zeros(2, 5, 8), torch.zeros(2, 8), torch.zeros(2, 8)
    q, t, lse, pos = torch.zeros(1, 2, 5, 8), torch.zeros(1, 2, 8), torch.zeros(1, 2, 5), torch.zeros(1, dtype=torch.int64)
    c = torch.zeros(1, 2, 4, 8)
    return {
        "gated_workspace": lambda s: hla.gated_workspace(x, stream=s),
        "gated_forward": lambda s: hla.gated_forward(x, x, stream=s),
        "gated_backward": lambda s: hla.gated_backward(x, x, x, x, stream=s),
        "gated_step": lambda s: hla.gated_step(state, row, row, stream=s),
        "window_forward": lambda s: hla.window_forward(q, q, q, 3, stream=s),
        "window_workspace": lambda s: hla.window_workspace(q, q, q, 3, stream=s),
        "window_backward": lambda s: hla.window_backward(q, q, q, q, lse, q, 3, stream=s),
        "window_cache_fill": lambda s: hla.window_cache_fill(c, c.clone(), q, q, 4, stream=s),
        "window_step": lambda s: hla.window_step(c, c.clone(), pos, t, t, t, 4, stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_stream_of_another_device(name, monkeypatch):
    monkeypatch.setattr(hla, "_current", lambda t: t.device)  # CPU tensors stand in for those of the current device
    stream = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        calls()[name](stream)
