"""The selective state space scan on the CUDA cores over more chunks than one span holds: the same
bits as each sequence alone, which fits one."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
from test_ssm_gpu import ARGS, BF16, F32, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,H,n,P,N,L", [(F32, 8, 64, 600, 64, 64, (600, 0, 1, 320, 321, 599, 64, 400)), (BF16, 8, 64, 600, 63, 64, None),
                                               (F32, 8, 16, 700, 128, 128, (700, 352, 351, 0, 353, 32, 640, 1)), (BF16, 3, 1400, 130, 40, 64, None)])
def test_spans_give_what_one_span_gives(dtype, B, H, n, P, N, L):
    c = inputs(B, H, H, n, P, N, dtype, seed=n)
    L = None if L is None else torch.tensor(L, dtype=torch.int32, device="cuda")
    kw = dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=True)

    def run(s):
        a = [c[k] if k == "A" else c[k][s] for k in ARGS]
        k = dict(kw, state_in=c["state"][s], lengths=None if L is None else L[s])
        y, st = hla.ssm_forward(*a, return_state=True, **k)
        r = hla.ssm_backward(*a, c["dy"][s], d_state_out=c["dstate"][s], want_dstate=True, **k)
        return y, st, r.dx, r.d_dt, r.dB, r.dC, r.d_state_in

    rows = run(slice(0, B))
    alone = [run(slice(b, b + 1)) for b in range(B)]
    hla.hla_sync_status()
    for i, t in enumerate(rows):
        assert torch.equal(t, torch.cat([a[i] for a in alone])), i


def test_groups_over_spans():
    """Heads that share B and C, whose gradients are joined span by span."""
    check(inputs(6, 100, 10, 520, 64, 64, F32, seed=1), torch.tensor([520, 3, 0, 448, 449, 260], dtype=torch.int32, device="cuda"))


def test_a_bounded_workspace_is_all_that_a_prompt_takes():
    B, H, n, P, N = 1, 64, 16384, 64, 128
    x, dt = torch.zeros(B, H, n, P, dtype=BF16, device="cuda"), torch.zeros(B, H, n, dtype=BF16, device="cuda")
    b, A = torch.zeros(B, 1, n, N, dtype=BF16, device="cuda"), -torch.ones(H, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y = hla.ssm_forward(x, dt, A, b, b)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 2 * y.numel() * 2
