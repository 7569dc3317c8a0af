"""Rates of 4 to 30: gates of e^-4 to e^-30, whose relative error reaches d_state_in, dg, d_rate
and, where x is zero, y.  Bounds: with g >= 0 sigma(g) comes out within 6 half steps of fp32 (its exponential
within |g| + 5 of them times 1 - sigma, the quotient within 3), r sigma(g) within 7, so exp of it within 8 for
each unit of r sigma(g), and within the four of the exponential itself, which the 32 cover."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import constant_state_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("rate", [4.0, 8.0, 16.0, 30.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,n,d", [(2, 1, 64), (2, 2, 33), (1, 200, 48), (2, 2, 1280), (1, 300, 2560)])
def test_fast_channels(B, n, d, dtype, rate, zeros, monkeypatch):
    monkeypatch.setattr(ref, "K_GATE", 32 + 8 * rate)
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    g, dy, st, ds = r(B, n, d).abs().to(dtype), r(B, n, d).to(dtype), r(B, d), r(B, d)
    x = torch.zeros_like(g) if zeros else r(B, n, d).to(dtype)
    if zeros:
        dy = torch.zeros_like(dy)
    rates = torch.full((d,), rate, device="cuda")
    y, s = hla.gated_forward(x, g, "rate", rates, state_in=st, return_state=True)
    q = hla.gated_backward(x, g, y, dy, "rate", rates, state_in=st, d_state_out=ds, want_dstate=True)
    hla.hla_sync_status()
    ry, rs, Ey, Es = ref.gated_forward(x, g, "rate", rates, st)
    ref.close(y, ry, Ey, "y")
    ref.close(s, rs, Es, "state_out")
    for name, want in ref.gated_backward(x, g, y, dy, "rate", rates, st, ds).items():
        ref.close(getattr(q, name), *want, name)
    if n == 1:
        nxt, out = torch.empty_like(st), torch.empty_like(x[:, 0])
        hla.gated_step(st, x[:, 0], g[:, 0], "rate", rates, state_out=nxt, out=out)
        ref.close(out, ry[:, 0], Ey[:, 0], "step's y")
        ref.close(nxt, rs, Es, "step's state")
