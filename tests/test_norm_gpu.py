"""Norm over groups of channels with an activation (hla_norm_forward, _backward) against its
64-bit form."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MODES = [("none", "none"), ("none", "silu"), ("after", "silu"), ("before", "silu")]


def inputs(B, n, d, dtype, seed=0, mean=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=(r(B, n, d) + mean).to(dtype), gate=r(B, n, d).to(dtype), weight=1 + 0.3 * r(d), bias=r(d), dy=r(B, n, d).to(dtype))


def close(got, want, name):
    val, e = want
    ref.close(got, val, e + (ref.half_step(got.dtype) * (val.abs() + e) if got.dtype == BF16 else 2 * ref.U * val.abs()), name)


def check(c, groups, gate, act, center, lengths=None, affine=True, eps=1e-5, out=None, grads=None):
    z = c["gate"] if gate != "none" else None
    w, b = (c["weight"], c["bias"]) if affine else (None, None)
    kw = dict(groups=groups, eps=eps, center=center, gate=z, gate_first=gate == "before", activation=act, lengths=lengths)
    want = ref.norm(c["x"], w, b, groups, eps, center, z, gate == "before", act, lengths, c["dy"])
    y = hla.norm_forward(c["x"], w, b, out=out, **kw)
    r = hla.norm_backward(c["x"], c["dy"], w, b, out=grads, **kw)
    hla.hla_sync_status()
    close(y, want["y"], "y")
    close(r.dx, want["dx"], "dx")
    assert (r.d_gate is not None) == (z is not None) and (r.d_weight is not None) == affine
    for name in (("d_gate",) if z is not None else ()) + (("d_weight", "d_bias") if affine else ()):
        close(getattr(r, name), want[name], name)
    return y, r


@pytest.mark.parametrize("gate,act", MODES)
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,n,d,groups", [(1, 1, 8, 1), (2, 3, 64, 4), (1, 5, 30, 3), (2, 33, 520, 65), (1, 40, 192, 2)])
def test_forward_and_gradients(B, n, d, groups, dtype, center, gate, act):
    check(inputs(B, n, d, dtype, seed=n + d), groups, gate, act, center)


@pytest.mark.parametrize("m", [63, 64, 65, 120, 128, 129, 256, 257, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4095, 4096, 4104, 8192])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_widths_of_a_group(m, dtype):
    """Both sides of every team size, whole and odd."""
    check(inputs(2, 7, 2 * m, dtype, seed=m), 2, "after", "silu", True)
    check(inputs(1, 7, m, dtype, seed=m), 1, "before", "silu", False)


@pytest.mark.parametrize("gate,act", MODES)
def test_groups_wider_than_a_team_holds(gate, act):
    check(inputs(2, 3, 2 * 8200, BF16), 2, gate, act, True)
    check(inputs(1, 2, 9001, F32), 1, gate, act, False)


@pytest.mark.parametrize("d,groups", [(64, 1), (50, 5), (8 * 300, 300)])
def test_padded_batch(d, groups):
    n = 41
    c = inputs(6, n, d, BF16, seed=3)
    L = torch.tensor([n, 0, 1, 20, n + 9, -4], dtype=torch.int32, device="cuda")
    dead = ~ref.live_rows(L, 6, n, "cuda")[..., None].expand(-1, -1, d)
    for k in ("x", "dy", "gate"):
        c[k] = torch.where(dead, torch.full_like(c[k], float("nan")), c[k])
    zero = lambda t: torch.where(dead, torch.zeros_like(t), t)  # noqa: E731
    kw = dict(groups=groups, gate=c["gate"], activation="silu", lengths=L)
    y = hla.norm_forward(c["x"], c["weight"], c["bias"], out=torch.full_like(c["x"], 7.0), **kw)
    r = hla.norm_backward(c["x"], c["dy"], c["weight"], c["bias"], out=(torch.full_like(y, 7.0), torch.full_like(y, 7.0)), **kw)
    hla.hla_sync_status()
    assert all(bool((t[dead] == 7).all()) for t in (y, r.dx, r.d_gate))
    want = ref.norm(zero(c["x"]), c["weight"], c["bias"], groups, 1e-5, True, zero(c["gate"]), False, "silu", L, zero(c["dy"]))
    for name, t in (("y", zero(y)), ("dx", zero(r.dx)), ("d_gate", zero(r.d_gate)), ("d_weight", r.d_weight), ("d_bias", r.d_bias)):
        close(t, want[name], name)
    y, r = hla.norm_forward(c["x"], **kw), hla.norm_backward(c["x"], c["dy"], **kw)
    assert not any(bool(t[dead].any()) for t in (y, r.dx, r.d_gate))


@pytest.mark.parametrize("rows", [151, 153, 305, 700])
def test_rows_behind_the_first_of_each_cta(rows):
    check(inputs(1, rows, 96, BF16, seed=rows), 2, "after", "silu", True)


@pytest.mark.parametrize("gate,act", MODES)
@pytest.mark.parametrize("d,groups,dtype", [(4096, 1, BF16), (1024, 1, F32), (520, 5, BF16)])
def test_many_rows_of_each_cta(d, groups, dtype, gate, act):
    """Rows that come ahead of their turn, dead ones between them left out."""
    n = 700
    L = torch.tensor([n, 333, n - 1], dtype=torch.int32, device="cuda")
    check(inputs(3, n, d, dtype, seed=d), groups, gate, act, False, L)


@pytest.mark.parametrize("layout", ["slice", "time_major", "odd_offset", "broadcast"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(layout, dtype):
    B, n, d = 2, 50, 96
    c = inputs(B, n, d, dtype, seed=9)
    out = grads = None
    if layout == "slice":
        wide = torch.cat([c["x"], c["gate"]], -1)
        c["x"], c["gate"] = wide[..., :d], wide[..., d:]
        both = torch.zeros(B, n, 3 * d, dtype=dtype, device="cuda")
        out, grads = both[..., :d], (both[..., d:2 * d], both[..., 2 * d:])
    elif layout == "time_major":
        c["x"] = c["x"].transpose(0, 1).contiguous().transpose(0, 1)
        out = torch.zeros(n, B, d, dtype=dtype, device="cuda").transpose(0, 1)
    elif layout == "odd_offset":
        flat = torch.zeros(B * n * d + 1, dtype=dtype, device="cuda")
        flat[1:] = c["gate"].reshape(-1)
        c["gate"] = flat[1:].view(B, n, d)
    else:
        c["gate"], c["dy"] = c["gate"][:1].expand(B, n, d), c["dy"][:, :1].expand(B, n, d)
    check(c, 4, "after", "silu", True, out=out, grads=grads)


def test_without_scale_and_shift():
    check(inputs(2, 9, 64, BF16), 2, "none", "none", True, affine=False)


def test_far_mean_and_zero_rows():
    """A mean of 100 deviations; rows of equal values, whose deviation is eps alone."""
    check(inputs(1, 20, 256, F32, mean=100.0), 1, "none", "none", True)
    c = inputs(1, 4, 64, F32)
    c["x"] = torch.full_like(c["x"], 0.5)
    check(c, 1, "none", "silu", True, eps=1e-3)
    c["x"] = torch.zeros_like(c["x"])
    check(c, 2, "after", "silu", False, eps=1e-3)


def test_no_tokens():
    x, w = torch.zeros(2, 0, 32, device="cuda"), torch.ones(32, device="cuda")
    assert hla.norm_forward(x, w).shape == x.shape
    r = hla.norm_backward(x, x, w, w)
    assert not bool(r.d_weight.any()) and not bool(r.d_bias.any())


def test_same_bits_and_shared_workspace():
    c, o = inputs(2, 700, 320, BF16), inputs(1, 500, 320, BF16, seed=1)
    ws = hla.norm_workspace(c["x"])
    run = lambda c, g: hla.norm_backward(c["x"], c["dy"], c["weight"], c["bias"], groups=g, workspace=ws)  # noqa: E731
    a = run(c, 5)
    run(o, 40)
    b = run(c, 5)
    assert torch.equal(a.dx, b.dx) and torch.equal(a.d_weight, b.d_weight) and torch.equal(a.d_bias, b.d_bias)


def test_gradient_against_differences():
    c = inputs(1, 3, 16, F32)
    f = lambda x: (hla.norm_forward(x, c["weight"], c["bias"], 2, 0.5, gate=c["gate"], activation="silu").double() * c["dy"].double()).sum()  # noqa: E731
    r = hla.norm_backward(c["x"], c["dy"], c["weight"], c["bias"], 2, 0.5, gate=c["gate"], activation="silu")
    e = torch.randn_like(c["x"])
    e = e / e.norm()
    h = 1e-2
    got, want = float((f(c["x"] + h * e) - f(c["x"] - h * e)) / (2 * h)), float((r.dx * e).sum())
    # z's third derivative along a unit step is below 15 / eps^1.5 of z's spread (43); rounding 1e-5 / h
    size = float(((c["weight"] * c["gate"]).abs() * c["dy"].abs()).sum()) * 43
    assert abs(got - want) <= h * h / 6 * size + 2e-3
