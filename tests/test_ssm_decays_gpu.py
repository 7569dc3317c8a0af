"""Decays of the selective state space scan: how exactly they are formed."""
import math

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def bound(d):
    """Relative error of dt 2^-d, d the sum of log decays between two tokens of a chunk, in units of
    u = 2^-24.  The exponent: A log2(e) is rounded twice and its product with dt once, 3 d u; each of the
    two running sums' remainders, below one half, is rounded at most nine times (three additions of a
    lane's tokens, five of the lanes, one of both) by u / 2, 9 u for both; their difference, below
    one, by u, and its sum with the whole numbers by u max(1, d).  ex2 is 4 u off, the products with dt, x and
    the weight round four times."""
    return ref.U * (math.log(2) * (3 * d + 10 + d.clamp(min=1)) + 8)


def impulses(n, dtype, seed):
    """Head h of n has its only input at token h; steps of 0.29 to 0.46 in the decays' exponent."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = (0.2 + 0.12 * torch.rand(1, 1, n, generator=gen, device="cuda")).to(dtype).expand(1, n, n)
    return dt, torch.eye(n, device="cuda", dtype=dtype)[None], torch.full((n,), -1.0, device="cuda")


@pytest.mark.parametrize("seed", range(4))
def test_decays_between_tokens_on_the_cuda_cores(seed):
    n = 64
    dt, x, A = impulses(n, F32, seed)
    one = torch.ones(1, 1, n, 1, device="cuda")
    y = hla.ssm_forward(x[..., None], dt, A, one, one)[0, :, :, 0].double()  # [input's token][output's]
    s = dt[0, 0].double().cumsum(0)
    e = s[None, :] - s[:, None]
    off = (y / (dt[0, 0].double()[:, None] * torch.exp(-e)) - 1).abs()
    late = torch.ones(n, n, device="cuda").triu().bool()
    assert not bool(y[~late].any())
    assert bool((off <= bound(e / math.log(2)))[late].all()), float(off[late].max())


@pytest.mark.parametrize("seed", range(4))
def test_decays_to_a_chunks_end_on_the_tensor_cores(seed):
    n = 128
    dt, x, A = impulses(n, BF16, seed)
    x = torch.nn.functional.pad(x[..., None], (0, 7))
    one = torch.zeros(1, 1, n, 8, device="cuda", dtype=BF16)
    one[..., 0] = 1
    st = hla.ssm_forward(x, dt, A, one, one, return_state=True)[1]
    hla.hla_sync_status()
    s = dt[0, 0].double().cumsum(0)
    e = s[-1] - s
    off = (st[0, :, 0, 0].double() / (dt[0, 0].double() * torch.exp(-e)) - 1).abs()
    assert bool((off <= bound(e / math.log(2))).all()), float(off.max())
