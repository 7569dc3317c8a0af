"""Long chains of few channels whose gates keep everything: each tile's state is the sum of
all tiles before it, so a look-back that starts or folds wrongly shows.  All values are whole
numbers below 2^24, exact in fp32 in any order of addition."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d", [(32768, 64), (32768, 33), (32767, 32), (32768, 2), (65536, 16)])
def test_running_sums_are_exact(n, d, dtype):
    one = torch.ones(1, n, d, dtype=dtype, device="cuda")
    state = torch.arange(d, dtype=F32, device="cuda")[None]
    t = torch.arange(n, dtype=F32, device="cuda")[None, :, None]
    h = t + 1 + state[:, None]                  # after token t
    gh = n - t + 2 * state[:, None]             # gradient of h_t: dy of ones, d_state of 2 state
    y_want, dx_want = h.to(dtype), gh.to(dtype)
    before = torch.cat([state[:, None], y_want[:, :-1].float()], 1)
    dg_want = (gh * before).to(dtype)
    ws = hla.gated_workspace(one)
    for i in range(50):
        y, s = hla.gated_forward(one, one, state_in=state, return_state=True, workspace=ws)
        assert torch.equal(s, n + state), i
        assert torch.equal(y, y_want), i
        r = hla.gated_backward(one, one, y, one, state_in=state, d_state_out=2 * state, want_dstate=True, workspace=ws)
        assert torch.equal(r.d_state_in, n + 2 * state), i
        assert torch.equal(r.dx, dx_want) and torch.equal(r.dg, dg_want), i
    hla.hla_sync_status()


def test_gates_that_nearly_keep_everything():
    """Against the recurrence in 64 bits, with gates of 1 - 2^-12: a few thousand tokens count."""
    n, d, a = 32768, 64, 1 - 2.0 ** -12
    x = torch.randn(1, n, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    g = torch.full_like(x, a)
    h, want = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.empty(n, d, dtype=torch.float64, device="cuda")
    H = h.clone()
    for t in range(n):
        h = a * h + x[0, t].double()
        H = a * H + x[0, t].double().abs()
        want[t] = h
    # each token rounds the state once, and a tile's map and the fold once more; all of it decays with a
    most = 4 * 2.0 ** -24 * float(H.max()) / (1 - a)
    first = None
    for i in range(20):
        y = hla.gated_forward(x, g)
        assert float((y[0].double() - want).abs().max()) <= most, i
        first = y if first is None else first
        assert torch.equal(y, first), i
    hla.hla_sync_status()
