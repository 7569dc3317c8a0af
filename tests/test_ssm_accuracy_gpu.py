"""How far the selective state space scan is off in 2-norms.  The tensor-core path in the forms that
training and prefill give it: many heads of a group through one CTA, with and without parts of dB
and dC to add up, both numbers of column tiles, several pieces of a head.

Bounds.  A value rounded to bf16 is off by 2^-8 / sqrt(3) of its power of two in the mean square; over mantissas
spread over their logarithm that is 1.66e-3 of the value.  Outputs in bf16 are rounded when stored; y, dx, dB
and dC also take a weight or a state rounded once.  Two such roundings in quadrature: 2.35e-3,
and 2.5e-3 leaves room for the scatter of a sample (a third rounding of as much would make 2.9e-3).
States and gradients of initial states are sums of exact products in fp32 with decays that are 2^-20
off (9.5e-7, all terms together at worst): 1.5e-6.  The gradients of A and dt_bias take sums over a chunk of 128 tokens and
their differences: about ten roundings of u = 2^-24 of a partial sum that is some 10 times the
difference, which do not add up from token to token: 5e-6.  dD: products and sums in fp32, 1e-6.
fp32: every output is such a sum, d_dt takes the differences.
dy is y and d_state_out the state, so that no gradient of A, D or dt_bias is what sums cancel to.
"""
import math

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref
from test_ssm_gpu import ARGS, BF16, F32, inputs

pytestmark = pytest.mark.gpu
BOUNDS = dict(y=2.5e-3, state=1.5e-6, dx=2.5e-3, dB=2.5e-3, dC=2.5e-3, d_dt=2.5e-3, dA=5e-6, d_dt_bias=5e-6, dD=1e-6, d_state_in=1.5e-6)
BOUNDS_F32 = dict(BOUNDS, y=1.5e-6, dx=1.5e-6, dB=1.5e-6, dC=1.5e-6, d_dt=5e-6)

# B, H, G, n, P, N, lengths: heads of a group per CTA of the gradients
CASES = [
    (40, 6, 1, 256, 64, 128, False),   # six, dB and dC written by the CTA
    (40, 6, 1, 256, 64, 128, True),    # the same, padded
    (80, 3, 1, 100, 128, 128, False),  # three of two column tiles, the same
    (110, 16, 1, 128, 32, 64, False),  # sixteen, states of one block
    (2, 8, 2, 1500, 64, 128, False),   # two, parts of dB and dC added up; several pieces
    (1, 5, 1, 2100, 128, 64, True),    # pieces in parts
]


def errors(dtype, B, H, G, n, P, N, ragged):
    c = inputs(B, H, G, n, P, N, dtype, seed=B + H)
    L = torch.tensor([n - 37 * i % n for i in range(B)], dtype=torch.int32, device="cuda") if ragged else None
    kw = dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=True, lengths=L)
    args = [c[k] for k in ARGS]
    y, s = hla.ssm_forward(*args, state_in=c["state"], return_state=True, **kw)
    r = hla.ssm_backward(*args, y, state_in=c["state"], d_state_out=s, want_dstate=True, **kw)
    hla.hla_sync_status()
    steps, slope = ref._steps(c["dt"], c["dt_bias"], True)
    want = ref._scan(c["x"], steps, slope, *args[2:], c["D"], c["state"], L, y, s, False)
    got = dict(r._asdict(), y=y, state=s)
    return {k: float((got[k].double() - want[k]).norm() / want[k].norm()) for k in BOUNDS}


@pytest.mark.parametrize("B,H,G,n,P,N,ragged", CASES)
def test_on_the_tensor_cores(B, H, G, n, P, N, ragged):
    e = errors(BF16, B, H, G, n, P, N, ragged)
    assert all(math.isfinite(e[k]) and e[k] <= BOUNDS[k] for k in e), e


@pytest.mark.parametrize("B,H,G,n,P,N,ragged", [(2, 8, 2, 700, 64, 128, False), (3, 6, 2, 300, 48, 40, True), (1, 3, 1, 500, 128, 128, False)])
def test_in_fp32(B, H, G, n, P, N, ragged):
    e = errors(F32, B, H, G, n, P, N, ragged)
    assert all(math.isfinite(e[k]) and e[k] <= BOUNDS_F32[k] for k in e), e
