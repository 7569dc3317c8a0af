"""Selective state space scan (hla_ssm_forward, _backward, _step) against its 64-bit form."""
import math

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def inputs(B, H, G, n, P, N, dtype, softplus=True, seed=0, rates=(1.0, 16.0), steps=(0.001, 0.1)):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    at = torch.exp(u(H) * math.log(steps[1] / steps[0]) + math.log(steps[0]))
    dt = 0.5 * r(B, H, n) if softplus else at[:, None] * torch.exp(0.5 * r(B, H, n))
    return dict(x=r(B, H, n, P).to(dtype), dt=dt.to(dtype), A=-(rates[0] + (rates[1] - rates[0]) * u(H)), B=r(B, G, n, N).to(dtype),
                C=r(B, G, n, N).to(dtype), D=r(H), dt_bias=at + torch.log(-torch.expm1(-at)) if softplus else None, dt_softplus=softplus,
                state=r(B, H, N, P), dy=r(B, H, n, P).to(dtype), dstate=r(B, H, N, P))


def tensor_cores(c):
    """Whether a bf16 call may round its operands to bf16: any that is not fp32."""
    return c["x"].dtype == BF16


def close(got, want, name):
    val, e = want
    ref.close(got, val, e + (ref.half_step(got.dtype) * (val.abs() + e) if got.dtype == BF16 else 2 * ref.U * val.abs()), name)


ARGS = ("x", "dt", "A", "B", "C")


def run(c, lengths=None, state=True, out=None, grads=None, ws=None, bws=None):
    st, ds = (c["state"], c["dstate"]) if state else (None, None)
    kw = dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=c["dt_softplus"], lengths=lengths)
    y, s = hla.ssm_forward(*(c[k] for k in ARGS), state_in=st, return_state=True, out=out, workspace=ws, **kw)
    r = hla.ssm_backward(*(c[k] for k in ARGS), c["dy"], state_in=st, d_state_out=ds, want_dstate=True, out=grads, workspace=bws, **kw)
    hla.hla_sync_status()
    return y, s, r


def check(c, lengths=None, state=True, **kw):
    st, ds = (c["state"], c["dstate"]) if state else (None, None)
    y, s, r = run(c, lengths, state, **kw)
    want = ref.ssm(*(c[k] for k in ARGS), c["D"], c["dt_bias"], c["dt_softplus"], st, lengths, c["dy"], ds, tensor_cores(c))
    close(y, want["y"], "y")
    close(s, want["state"], "state_out")
    assert (r.dD is not None) == (c["D"] is not None) and (r.d_dt_bias is not None) == (c["dt_bias"] is not None)
    for name in r._fields:
        if getattr(r, name) is not None:
            close(getattr(r, name), want[name], name)
    return y, s, r


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,G,n,P,N", [(1, 1, 1, 1, 1, 1), (2, 2, 1, 2, 8, 16), (1, 3, 3, 31, 5, 7), (1, 2, 1, 64, 64, 64), (2, 4, 2, 65, 32, 128),
                                         (1, 2, 2, 127, 64, 40), (1, 3, 1, 128, 64, 128), (1, 2, 1, 129, 128, 128), (2, 6, 2, 300, 48, 40),
                                         (1, 1, 1, 520, 64, 128), (1, 4, 1, 200, 128, 16), (1, 2, 1, 150, 72, 104)])
def test_forward_and_gradients(B, H, G, n, P, N, dtype, softplus):
    check(inputs(B, H, G, n, P, N, dtype, softplus, seed=n + P))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_states_skip_and_bias(dtype):
    c = inputs(2, 4, 2, 150, 64, 64, dtype)
    c["D"] = c["dt_bias"] = None
    check(c, state=False)


@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (BF16, 64, 64), (BF16, 12, 20), (F32, 64, 64), (F32, 128, 128)])
@pytest.mark.parametrize("n", [1, 130, 290])
def test_padded_batch(n, P, N, dtype):
    """Lengths of n, 0, 1, half, one chunk, and beyond both ends; what lies behind them is not read."""
    c = inputs(7, 2, 1, n, P, N, dtype, seed=5)
    L = torch.tensor([n, 0, 1, n // 2, min(n, 128), n + 9, -4], dtype=torch.int32, device="cuda")
    dead = ~ref.live_rows(L, 7, n, "cuda")[:, None]
    clean = dict(c)
    for k in ("x", "dy", "B", "C", "dt"):
        d = dead if k == "dt" else dead[..., None]
        clean[k] = torch.where(d, torch.zeros_like(c[k]), c[k])
        c[k] = torch.where(d, torch.full_like(c[k], float("nan")), c[k])
    seven = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    y, s, r = run(c, L, out=seven(c["x"]), grads=tuple(seven(c[k]) for k in ("x", "dt", "B", "C")))
    want = ref.ssm(*(clean[k] for k in ARGS), c["D"], c["dt_bias"], True, c["state"], L, clean["dy"], c["dstate"], tensor_cores(c))
    for name, t in (("y", y), ("dx", r.dx), ("d_dt", r.d_dt), ("dB", r.dB), ("dC", r.dC)):
        d = dead.expand_as(t) if t.dim() == 3 else dead[..., None].expand_as(t)
        assert bool((t[d] == 7).all()), name
        close(torch.where(d, torch.zeros_like(t), t), want[name], name)
    close(s, want["state"], "state_out")
    for name in ("dA", "dD", "d_dt_bias", "d_state_in"):
        close(getattr(r, name), want[name], name)


def test_new_outputs_of_a_padded_batch_are_zero_behind_the_lengths():
    c = inputs(2, 2, 1, 150, 64, 64, BF16)
    L = torch.tensor([150, 7], dtype=torch.int32, device="cuda")
    y, _, r = run(c, L)
    assert not any(bool(t[1, :, 7:].any()) for t in (y, r.dx, r.d_dt, r.dB, r.dC))


@pytest.mark.parametrize("layout", ["channels_last", "broadcast", "odd_offset", "odd_stride", "time_major"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(layout, dtype):
    B, H, G, n, P, N = 2, 4, 2, 200, 64, 64
    c = inputs(B, H, G, n, P, N, dtype, seed=9)
    out = grads = None
    if layout == "channels_last":  # x, B and C side by side in one projection, their gradients too
        def parts(wide):
            f = lambda a, h, w: wide[..., a:a + h * w].unflatten(-1, (h, w)).transpose(1, 2)  # noqa: E731
            return f(0, H, P), f(H * P, G, N), f(H * P + G * N, G, N)
        t = lambda k: c[k].transpose(1, 2).flatten(2)  # noqa: E731
        c["x"], c["B"], c["C"] = parts(torch.cat([t("x"), t("B"), t("C")], -1))
        c["dt"] = c["dt"].transpose(1, 2).contiguous().transpose(1, 2)
        dx, dB, dC = parts(torch.zeros(B, n, H * P + 2 * G * N, dtype=dtype, device="cuda"))
        grads = dx, torch.zeros_like(c["dt"]), dB, dC
        y, _, _ = run(c)
        assert y.transpose(1, 2).is_contiguous()
    elif layout == "broadcast":    # one dt for the heads, one x for the batch, dy of a sum over tokens
        c["dt"] = c["dt"][:, :1].expand(B, H, n)
        c["x"], c["dy"] = c["x"][:1].expand(B, H, n, P), c["dy"][:, :, :1].expand(B, H, n, P)
    elif layout == "odd_offset":
        flat = torch.zeros(B * G * n * N + 1, dtype=dtype, device="cuda")
        flat[1:] = c["B"].reshape(-1)
        c["B"] = flat[1:].view(B, G, n, N)
    elif layout == "odd_stride":
        wide = torch.zeros(B, H, n, P + 1, dtype=dtype, device="cuda")
        wide[..., :P] = c["x"]
        c["x"] = wide[..., :P]
        out = torch.zeros(B, H, n, P + 3, dtype=dtype, device="cuda")[..., :P]
    else:
        c["x"] = c["x"].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
        out = torch.zeros(n, B, H, P, dtype=dtype, device="cuda").permute(1, 2, 0, 3)
    check(c, out=out, grads=grads)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rates,steps", [((1e-4, 1e-3), (0.001, 0.1)), ((50.0, 100.0), (0.5, 2.0)), ((1.0, 1.0), (1e-6, 1e-5))])
def test_slow_and_steep_decays(rates, steps, dtype):
    check(inputs(1, 2, 1, 300, 64, 64, dtype, False, rates=rates, steps=steps))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_resets(dtype):
    """Tokens whose decay forgets everything (2^-256 and beyond), others that keep everything."""
    c = inputs(1, 2, 1, 260, 64, 64, dtype, False)
    dt = torch.zeros(1, 2, 260, device="cuda")
    dt[..., ::37] = 1e4
    dt[..., 1::5] = 0.01
    c["dt"] = dt.to(dtype)
    check(c)


def test_growing_states():
    """A > 0: the state grows, by at most 2^14 here."""
    c = inputs(1, 2, 1, 200, 64, 64, F32, False)
    c["A"] = c["A"].abs() / 16
    c["dt"] = c["dt"].clamp(max=0.05)
    check(c)


@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (BF16, 64, 64), (BF16, 128, 16), (BF16, 33, 20), (F32, 48, 40), (F32, 128, 128)])
@pytest.mark.parametrize("B,H,G", [(1, 2, 1), (3, 4, 2), (32, 16, 1)])
def test_steps_continue_a_prompt(B, H, G, dtype, P, N):
    c = inputs(B, H, G, 24, P, N, dtype, seed=2)
    kw = dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=True)
    y0, st = hla.ssm_forward(*(c[k][..., :20] if k == "dt" else c[k][:, :, :20] if k != "A" else c[k] for k in ARGS),
                             state_in=c["state"], return_state=True, **kw)
    got = [y0]
    for t in range(20, 24):
        got.append(hla.ssm_step(st, *(c[k] if k == "A" else c[k][:, :, t] for k in ARGS), **kw)[:, :, None])
    hla.hla_sync_status()
    want = ref.ssm(*(c[k] for k in ARGS), c["D"], c["dt_bias"], True, c["state"], tensor_cores=tensor_cores(c))
    close(torch.cat(got, 2), want["y"], "y")
    close(st, want["state"], "state")


def test_idle_sequences_of_a_step():
    c = inputs(4, 2, 1, 1, 64, 64, BF16)
    live = torch.tensor([1, 0, 5, -1], dtype=torch.int32, device="cuda")
    st, out = c["state"].clone(), torch.full((4, 2, 64), 7.0, dtype=BF16, device="cuda")
    kw = dict(D=c["D"], dt_bias=c["dt_bias"], dt_softplus=True, lengths=live)
    args = [c[k] if k == "A" else c[k][:, :, 0] for k in ARGS]
    y = hla.ssm_step(st, *args, out=out, **kw)
    idle = live <= 0
    assert bool((y[idle] == 7).all()) and torch.equal(st[idle], c["state"][idle])
    want = ref.ssm(*(c[k] for k in ARGS), c["D"], c["dt_bias"], True, c["state"])
    close(y[~idle], tuple(t[:, :, 0][~idle] for t in want["y"]), "y")
    close(st[~idle], tuple(t[~idle] for t in want["state"]), "state")
    assert not bool(hla.ssm_step(st, *args, **kw)[idle].any())


def test_no_tokens():
    c = inputs(2, 2, 1, 3, 64, 64, BF16)
    for k in ("x", "B", "C", "dy", "dt"):
        c[k] = c[k][:, :, :0]
    y, s, r = run(c)
    assert y.shape == c["x"].shape and torch.equal(s, c["state"]) and torch.equal(r.d_state_in, c["dstate"])
    assert not any(bool(t.any()) for t in (r.dA, r.dD, r.d_dt_bias))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_same_bits_and_shared_workspace(dtype):
    """Another problem in between on the same workspace, which starts with NaN in it."""
    c, o = inputs(2, 6, 2, 400, 64, 128, dtype), inputs(1, 6, 2, 300, 64, 128, dtype, seed=1)
    ws, bws = hla.ssm_workspace(c["x"], c["B"]), hla.ssm_workspace(c["x"], c["B"], backward=True)
    ws.fill_(255), bws.fill_(255)
    a = run(c, ws=ws, bws=bws)
    run(o, ws=ws, bws=bws)
    b = run(c, ws=ws, bws=bws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(p, q) for p, q in zip(a[2], b[2]))


def test_many_heads_share_a_group():
    check(inputs(1, 24, 1, 140, 64, 64, BF16, seed=4))
    check(inputs(1, 24, 2, 70, 32, 16, F32, seed=4))


@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (BF16, 72, 64), (F32, 40, 24)])
def test_long_sequences(dtype, P, N):
    """A head's chunks shared by several CTAs; lengths that end inside the first, a middle and the last share."""
    c = inputs(4, 1, 1, 2500, P, N, dtype, seed=6, rates=(0.05, 0.5))
    check(c, torch.tensor([2500, 90, 1100, 2433], dtype=torch.int32, device="cuda"))
    check(inputs(1, 2, 2, 2100, P, N, dtype, seed=7), state=False)


@pytest.mark.parametrize("B,H,n,lengths", [(1, 17, 1147, None), (5, 1, 3910, [3910, 3700, 2049, 1, 2100]), (3, 13, 2001, [2001, 385, 1500]),
                                           (3, 13, 2048, [0, 2048, 768])])
def test_pieces_in_parts(B, H, n, lengths):
    """Shares of a head's chunks whose sums are formed in parts, one way and both ways."""
    c = inputs(B, H, 1, n, 8, 16, BF16, seed=n, rates=(0.05, 0.5))
    check(c, lengths and torch.tensor(lengths, dtype=torch.int32, device="cuda"))


def test_gradient_against_differences():
    c = inputs(1, 2, 1, 70, 8, 8, F32)
    f = lambda dt: (hla.ssm_forward(c["x"], dt, c["A"], c["B"], c["C"], dt_bias=c["dt_bias"], dt_softplus=True).double() * c["dy"].double()).sum()  # noqa: E731
    r = hla.ssm_backward(c["x"], c["dt"], c["A"], c["B"], c["C"], c["dy"], dt_bias=c["dt_bias"], dt_softplus=True)
    e = torch.randn_like(c["dt"])
    h = 1e-2
    d1 = float((f(c["dt"] + h * e) - f(c["dt"] - h * e)) / (2 * h))
    d2 = float((f(c["dt"] + 2 * h * e) - f(c["dt"] - 2 * h * e)) / (4 * h))
    # the two steps' difference is three times the smaller one's error of second order; rounding 1e-4 / h
    assert abs(d1 - float((r.d_dt * e).sum())) <= abs(d1 - d2) + 2e-2
