"""Sizes that 32 bits do not hold are refused by the selective state space layer's calls, not cut to
their low bits."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
from causal_prefix_scan_gb300 import _build

LONG = (1 << 32) + 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def calls():
    one = torch.zeros(1)
    x, w = one.expand(1, LONG, 1), torch.zeros(1, 2)
    h, dt, b, A = one.expand(1, 1, LONG, 1), one.expand(1, 1, LONG), one.expand(1, 1, LONG, 1), -torch.ones(1)
    many = one.expand(LONG, 1, 1, 1)
    return {
        "conv_forward": lambda: hla.conv_forward(x, w),
        "conv_workspace": lambda: hla.conv_workspace(x, w),
        "conv_backward": lambda: hla.conv_backward(x, x, w),
        "conv_step": lambda: hla.conv_step(one.expand(LONG, 1, 1), one.expand(LONG, 1), w),
        "ssm_workspace": lambda: hla.ssm_workspace(h, b),
        "ssm_forward": lambda: hla.ssm_forward(h, dt, A, b, b),
        "ssm_backward": lambda: hla.ssm_backward(h, dt, A, b, b, h),
        "ssm_step": lambda: hla.ssm_step(many, many[..., 0], one.expand(LONG, 1), A, many[..., 0], many[..., 0]),
        "norm_forward": lambda: hla.norm_forward(x),
        "norm_workspace": lambda: hla.norm_workspace(x),
        "norm_backward": lambda: hla.norm_backward(x, x),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_size_beyond_32_bits(name, monkeypatch):
    monkeypatch.setattr(hla, "_current", lambda t: t.device)  # CPU tensors stand in for those of the current device
    reached = []
    for kernel in [k for k in vars(hla) if k.startswith(("hla_conv_", "hla_ssm_", "hla_norm_")) and not k.endswith(("params", "gradients"))]:
        monkeypatch.setattr(hla, kernel, lambda *a: reached.append(a) or 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: reached.append(a) or pytest.fail("something was allocated"))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        calls()[name]()
    assert not reached
