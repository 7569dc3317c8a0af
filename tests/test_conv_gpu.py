"""Short causal convolution (hla_conv_forward, _backward, _step) against its 64-bit form."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def inputs(B, n, d, w, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=r(B, n, d).to(dtype), weight=r(d, w), bias=r(d), state=r(B, w - 1, d).to(dtype), dy=r(B, n, d).to(dtype),
                dstate=r(B, w - 1, d).to(dtype))


def close(got, want, name):
    val, e = want
    ref.close(got, val, e + (ref.half_step(got.dtype) * (val.abs() + e) if got.dtype == BF16 else 2 * ref.U * val.abs()), name)


def check(c, kind, lengths=None, state=True, bias=True, out=None, dx=None):
    st, ds, b = (c["state"], c["dstate"]) + (c["bias"],) if state else (None, None, c["bias"])
    b = b if bias else None
    want = ref.conv(c["x"], c["weight"], b, kind, st, lengths, c["dy"], ds)
    y, s = hla.conv_forward(c["x"], c["weight"], b, kind, state_in=st, return_state=True, lengths=lengths, out=out)
    r = hla.conv_backward(c["x"], c["dy"], c["weight"], b, kind, state_in=st, d_state_out=ds, want_dstate=True, lengths=lengths,
                          out=dx)
    hla.hla_sync_status()
    close(y, want["y"], "y")
    assert torch.equal(s.double(), want["state"][0])
    for name in ("dx", "d_weight", "d_state_in") + (("d_bias",) if bias else ()):
        close(getattr(r, name), want[name], name)
    assert (r.d_bias is not None) == bias
    return y, s, r


@pytest.mark.parametrize("kind", ["none", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,n,d,w", [(1, 1, 1, 2), (2, 2, 3, 4), (3, 3, 8, 4), (1, 31, 64, 3), (2, 33, 260, 4), (1, 128, 40, 2),
                                     (2, 257, 36, 4), (1, 300, 1001, 3)])
def test_forward_and_gradients(B, n, d, w, dtype, kind):
    check(inputs(B, n, d, w, dtype, seed=n + d), kind)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_state_and_bias(dtype):
    check(inputs(2, 70, 24, 4, dtype), "silu", state=False, bias=False)


@pytest.mark.parametrize("n,d", [(1, 8), (5, 16), (300, 34)])
def test_padded_batch(n, d):
    """Lengths of n, 0, 1, 2, half, n - 1, and beyond both ends; what lies behind them is not read."""
    c = inputs(8, n, d, 4, BF16, seed=3)
    L = torch.tensor([n, 0, 1, 2, n // 2, n - 1, n + 9, -4], dtype=torch.int32, device="cuda")
    dead = ~ref.live_rows(L, 8, n, "cuda")[..., None].expand(-1, -1, d)
    for k in ("x", "dy"):
        c[k] = torch.where(dead, torch.full_like(c[k], float("nan")), c[k])
    zeros = {k: torch.where(dead, torch.zeros_like(c[k]), c[k]) for k in ("x", "dy")}
    y, s = hla.conv_forward(c["x"], c["weight"], c["bias"], "silu", state_in=c["state"], return_state=True, lengths=L,
                            out=torch.full_like(c["x"], 7.0))
    r = hla.conv_backward(c["x"], c["dy"], c["weight"], c["bias"], "silu", state_in=c["state"], d_state_out=c["dstate"],
                          want_dstate=True, lengths=L, out=torch.full_like(c["x"], 7.0))
    hla.hla_sync_status()
    assert bool((y[dead] == 7).all()) and bool((r.dx[dead] == 7).all())
    want = ref.conv(zeros["x"], c["weight"], c["bias"], "silu", c["state"], L, zeros["dy"], c["dstate"])
    close(torch.where(dead, torch.zeros_like(y), y), want["y"], "y")
    close(torch.where(dead, torch.zeros_like(y), r.dx), want["dx"], "dx")
    assert torch.equal(s.double(), want["state"][0])
    for name in ("d_weight", "d_bias", "d_state_in"):
        close(getattr(r, name), want[name], name)
    y = hla.conv_forward(c["x"], c["weight"], lengths=L)
    r = hla.conv_backward(c["x"], c["dy"], c["weight"], lengths=L)
    assert not bool(y[dead].any()) and not bool(r.dx[dead].any())


@pytest.mark.parametrize("layout", ["slice", "time_major", "odd_offset", "odd_stride", "broadcast"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(layout, dtype):
    B, n, d = 2, 90, 48
    c = inputs(B, n, d, 4, dtype, seed=9)
    out = dx = None
    if layout == "slice":
        wide = torch.cat([c["x"], c["dy"]], -1)
        c["x"], c["dy"] = wide[..., :d], wide[..., d:]
        both = torch.zeros(B, n, 2 * d, dtype=dtype, device="cuda")
        out, dx = both[..., :d], both[..., d:]
    elif layout == "time_major":
        c["x"] = c["x"].transpose(0, 1).contiguous().transpose(0, 1)
        out, dx = (torch.zeros(n, B, d, dtype=dtype, device="cuda").transpose(0, 1) for _ in range(2))
    elif layout == "odd_offset":
        flat = torch.zeros(B * n * d + 1, dtype=dtype, device="cuda")
        flat[1:] = c["x"].reshape(-1)
        c["x"] = flat[1:].view(B, n, d)
    elif layout == "odd_stride":
        wide = torch.zeros(B, n, d + 1, dtype=dtype, device="cuda")
        wide[..., :d] = c["dy"]
        c["dy"] = wide[..., :d]
    else:
        c["x"], c["dy"] = c["x"][:1].expand(B, n, d), c["dy"][:, :1].expand(B, n, d)
    check(c, "silu", out=out, dx=dx)


def test_long_runs():
    """Many rounds of tiles, where each warp takes more tokens."""
    c = inputs(57, 32761, 2, 4, BF16, seed=8)
    L = torch.randint(0, 32762, (57,), generator=torch.Generator().manual_seed(8), dtype=torch.int32)
    L[0], L[1] = 32761, 32767
    check(c, "silu", L.cuda())


def test_far_values():
    """Pre-activations from -1e4 to 1e4: the sigmoid's exponential overflows on one side."""
    c = inputs(1, 64, 8, 2, F32)
    c["x"] = torch.linspace(-1e4, 1e4, 512, device="cuda").view(1, 64, 8)
    check(c, "silu")


@pytest.mark.parametrize("dtype,d", [(BF16, 256), (BF16, 50), (F32, 33)])
@pytest.mark.parametrize("kind", ["none", "silu"])
def test_steps_continue_a_prompt(dtype, d, kind):
    """A prompt and then single tokens give the bits of one long prompt's y and state."""
    c = inputs(3, 40, d, 4, dtype, seed=2)
    y, s = hla.conv_forward(c["x"], c["weight"], c["bias"], kind, state_in=c["state"], return_state=True)
    y0, st = hla.conv_forward(c["x"][:, :30], c["weight"], c["bias"], kind, state_in=c["state"], return_state=True)
    got = [y0] + [hla.conv_step(st, c["x"][:, t], c["weight"], c["bias"], kind)[:, None] for t in range(30, 40)]
    assert torch.equal(s, st)
    want = ref.conv(c["x"], c["weight"], c["bias"], kind, c["state"])["y"]
    close(torch.cat(got, 1), want, "y")
    close(y, want, "y")


def test_idle_sequences_of_a_step():
    c = inputs(4, 1, 24, 3, BF16)
    live = torch.tensor([1, 0, 5, -1], dtype=torch.int32, device="cuda")
    st, out = c["state"].clone(), torch.full((4, 24), 7.0, dtype=BF16, device="cuda")
    y = hla.conv_step(st, c["x"][:, 0], c["weight"], c["bias"], "silu", lengths=live, out=out)
    idle = live <= 0
    assert bool((y[idle] == 7).all()) and torch.equal(st[idle], c["state"][idle])
    want = ref.conv(c["x"], c["weight"], c["bias"], "silu", c["state"])
    close(y[~idle], tuple(t[:, 0][~idle] for t in want["y"]), "y")
    assert torch.equal(st[~idle].double(), want["state"][0][~idle])
    assert not bool(hla.conv_step(st, c["x"][:, 0], c["weight"], lengths=live)[idle].any())


def test_no_tokens():
    c = inputs(2, 4, 24, 3, BF16)
    x = c["x"][:, :0]
    y, s = hla.conv_forward(x, c["weight"], c["bias"], state_in=c["state"], return_state=True)
    r = hla.conv_backward(x, x, c["weight"], c["bias"], d_state_out=c["dstate"], want_dstate=True)
    assert y.shape == x.shape and torch.equal(s, c["state"]) and torch.equal(r.d_state_in, c["dstate"])
    assert not bool(r.d_weight.any()) and not bool(r.d_bias.any())
    assert not bool(hla.conv_forward(x, c["weight"], return_state=True)[1].any())


def test_same_bits_and_shared_workspace():
    c, o = inputs(2, 700, 80, 4, BF16), inputs(1, 500, 80, 4, BF16, seed=1)
    ws = hla.conv_workspace(c["x"], c["weight"])
    run = lambda c: hla.conv_backward(c["x"], c["dy"], c["weight"], c["bias"], "silu", workspace=ws)  # noqa: E731
    a = run(c)
    run(o)
    b = run(c)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_gradient_against_differences():
    c = inputs(1, 9, 4, 3, F32)
    f = lambda w: (hla.conv_forward(c["x"], w, c["bias"], "silu").double() * c["dy"].double()).sum()  # noqa: E731
    r = hla.conv_backward(c["x"], c["dy"], c["weight"], c["bias"], "silu")
    e = torch.randn(4, 3, device="cuda")
    got = float((f(c["weight"] + 1e-2 * e) - f(c["weight"] - 1e-2 * e)) / 2e-2)
    want = float((r.d_weight * e).sum())
    # third derivatives: h^2 / 6 times at most 36 of |dy| (|e||x|)^3 (below 20 each); rounding 1e-5 / h
    size = float((c["dy"].abs().sum() * (e.abs().max() * 3 * c["x"].abs().max()) ** 3))
    assert abs(got - want) <= 1e-4 / 6 * size + 1e-3
