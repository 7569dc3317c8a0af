"""Decays of the selective state space scan: how exactly they are formed, and values of A and dt at
the borders of what they may be."""
import math

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref
from test_ssm_gpu import BF16, F32, check, inputs

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype,P", [(BF16, 64), (BF16, 9), (F32, 64)])
def test_a_rate_that_is_not_a_number_reaches_its_head(dtype, P):
    """... in the prompt, its gradients and a step, and no other head."""
    c = inputs(1, 4, 2, 150, P, 16, dtype)
    args, kw = [c[k] for k in ("x", "dt", "A", "B", "C")], dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=True)
    want = hla.ssm_forward(*args, state_in=c["state"], return_state=True, **kw)
    args[2] = args[2].clone()
    args[2][1] = float("nan")
    y, s = hla.ssm_forward(*args, state_in=c["state"], return_state=True, **kw)
    r = hla.ssm_backward(*args, c["dy"], state_in=c["state"], want_dstate=True, **kw)
    hla.hla_sync_status()
    assert bool(y[:, 1].isnan().all()) and bool(s[:, 1].isnan().all())
    for h in (0, 2, 3):
        assert torch.equal(y[:, h], want[0][:, h]) and torch.equal(s[:, h], want[1][:, h])
    assert r.dA.isnan().tolist() == [False, True, False, False] and bool(r.d_state_in[:, 1].isnan().all())
    st = c["state"].clone()
    hla.ssm_step(st, *(t if t is args[2] else t[:, :, 0] for t in args), **kw)
    assert bool(st[:, 1].isnan().all()) and not bool(st[:, [0, 2, 3]].isnan().any())


@pytest.mark.parametrize("dtype,P", [(BF16, 64), (BF16, 9), (F32, 64)])
@pytest.mark.parametrize("n", [1, 40, 128, 200])
def test_a_rate_of_minus_infinity_forgets(n, dtype, P):
    """Every token starts anew: what lies behind the last one of a chunk takes nothing away."""
    c = inputs(2, 2, 1, n, P, 16, dtype, softplus=False)
    c["A"] = torch.full((2,), -math.inf, device="cuda")
    L = torch.tensor([n, (n + 1) // 2], dtype=torch.int32, device="cuda")
    y, s = hla.ssm_forward(*(c[k] for k in ("x", "dt", "A", "B", "C")), state_in=c["state"], return_state=True, lengths=L)
    hla.hla_sync_status()
    for b in range(2):
        t = int(L[b]) - 1
        x, dt, bt = c["x"][b, :, t].double(), c["dt"][b, :, t].double(), c["B"][b, :, t].double()
        want = (dt[:, None] * bt)[..., None] * x[:, None]
        ref.close(s[b], want, 4 * ref.U * want.abs(), "state")


@pytest.mark.parametrize("signs", [False, True])
def test_growing_states_on_the_tensor_cores(signs):
    """A > 0, and steps of both signs: the decays add up to 2^14 at most."""
    c = inputs(1, 2, 1, 200, 64, 64, BF16, False)
    c["A"] = c["A"].abs() / 16
    c["dt"] = c["dt"].clamp(max=0.05)
    if signs:
        c["dt"] = torch.where(torch.arange(200, device="cuda") % 50 < 25, -c["dt"], c["dt"])
    check(c)


@pytest.mark.parametrize("dtype,P", [(BF16, 64), (BF16, 9), (F32, 64)])
def test_tokens_ahead_of_an_overflow(dtype, P):
    """Steps of 2^8 a token: the 17th leaves fp32's range, those ahead of it are as they would be alone."""
    c = inputs(1, 2, 1, 100, P, 16, dtype, False)
    c["A"] = torch.ones(2, device="cuda")
    c["dt"] = torch.full_like(c["dt"], 5.5)
    args = [c[k] for k in ("x", "dt", "A", "B", "C")]
    y = hla.ssm_forward(*args, state_in=c["state"], D=c["D"])
    short = [t if t is c["A"] else t[:, :, :12] for t in args]
    want = ref.ssm(*short, c["D"], None, False, c["state"], tensor_cores=dtype == BF16)["y"]
    hla.hla_sync_status()
    y = y[:, :, :12]
    ref.close(y, want[0], want[1] + ref.half_step(dtype) * (want[0].abs() + want[1]) + 2 * ref.U * want[0].abs(), "y")
