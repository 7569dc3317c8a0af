"""Gated linear recurrence (hla_gated_forward, _backward, _step) against its 64-bit form."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import constant_state_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
GATES = ("given", "sigmoid", "rate")


def inputs(B, n, d, gate, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    z = 2 * r(B, n, d) + 1
    return dict(x=r(B, n, d).to(dtype), g=(torch.sigmoid(z) if gate == "given" else z).to(dtype), gate=gate,
                rate=torch.rand(d, generator=gen, device="cuda") * 2 + 0.01 if gate == "rate" else None,
                state_in=r(B, d), dy=r(B, n, d).to(dtype), d_state=r(B, d))


def lengths_of(B, n, kind):
    if kind is None:
        return None
    L = [n, 0, 1, n // 2, max(n - 1, 0), 200]
    return torch.tensor([min(L[i % len(L)], n) for i in range(B)], dtype=torch.int32, device="cuda")


def check(c, lengths=None, state=True, **kw):
    st = c["state_in"] if state else None
    y, s = hla.gated_forward(c["x"], c["g"], c["gate"], c["rate"], state_in=st, return_state=True, lengths=lengths, **kw)
    hla.hla_sync_status()
    ry, rs, Ey, Es = ref.gated_forward(c["x"], c["g"], c["gate"], c["rate"], st, lengths)
    ref.close(y, ry, Ey, "y")
    ref.close(s, rs, Es, "state_out")
    ds = c["d_state"] if state else None
    r = hla.gated_backward(c["x"], c["g"], y, c["dy"], c["gate"], c["rate"], state_in=st, d_state_out=ds,
                           want_dstate=True, lengths=lengths, **kw)
    hla.hla_sync_status()
    want = ref.gated_backward(c["x"], c["g"], y, c["dy"], c["gate"], c["rate"], st, ds, lengths)
    for name, (val, bound) in want.items():
        ref.close(getattr(r, name), val, bound, name)
    assert (r.d_rate is not None) == (c["gate"] == "rate")
    return y, s, r


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,n,d", [(1, 1, 1), (2, 2, 3), (1, 15, 64), (3, 16, 33), (1, 127, 65), (2, 128, 64),
                                   (1, 129, 2), (2, 257, 96), (1, 1000, 130)])
def test_forward_and_gradients(B, n, d, gate, dtype):
    check(inputs(B, n, d, gate, dtype, seed=n + d))


@pytest.mark.parametrize("gate", GATES)
def test_without_states(gate):
    check(inputs(2, 200, 40, gate, BF16), state=False)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("n,d", [(1, 7), (130, 64), (500, 34)])
def test_padded_batch(n, d, gate):
    c = inputs(6, n, d, gate, BF16, seed=5)
    L = lengths_of(6, n, "mixed")
    dead = torch.arange(n, device="cuda")[None, :, None] >= L[:, None, None]
    for t in ("x", "g", "dy"):  # what lies behind a length is not read
        c[t] = torch.where(dead, torch.full_like(c[t], float("nan")), c[t])
    clean = {k: torch.where(dead, torch.zeros_like(c[k]), c[k]) for k in ("x", "g", "dy")}
    mark = torch.full_like(c["x"], 7.0)
    y, s = hla.gated_forward(c["x"], c["g"], gate, c["rate"], state_in=c["state_in"], return_state=True, lengths=L,
                             out=mark)
    ry, rs, Ey, Es = ref.gated_forward(clean["x"], clean["g"], gate, c["rate"], c["state_in"], L)
    assert bool((y[dead.expand_as(y)] == 7.0).all())
    ref.close(torch.where(dead, torch.zeros_like(y), y), ry, Ey, "y")
    ref.close(s, rs, Es, "state_out")
    yn = torch.where(dead, torch.full_like(y, float("nan")), y)
    outs = torch.full_like(y, 7.0), torch.full_like(y, 7.0)
    r = hla.gated_backward(c["x"], c["g"], yn, c["dy"], gate, c["rate"], state_in=c["state_in"],
                           d_state_out=c["d_state"], want_dstate=True, lengths=L, out=outs)
    hla.hla_sync_status()
    want = ref.gated_backward(clean["x"], clean["g"], torch.where(dead, torch.zeros_like(y), y), clean["dy"], gate,
                              c["rate"], c["state_in"], c["d_state"], L)
    for name, (val, bound) in want.items():
        got = getattr(r, name)
        if name in ("dx", "dg"):
            assert bool((got[dead.expand_as(got)] == 7.0).all())
            got = torch.where(dead, torch.zeros_like(got), got)
        ref.close(got, val, bound, name)


def test_new_outputs_of_a_padded_batch_are_zero_behind_the_lengths():
    c = inputs(2, 40, 8, "sigmoid", BF16)
    L = torch.tensor([40, 3], dtype=torch.int32, device="cuda")
    y = hla.gated_forward(c["x"], c["g"], "sigmoid", lengths=L)
    r = hla.gated_backward(c["x"], c["g"], y, c["dy"], "sigmoid", lengths=L)
    assert not bool(y[1, 3:].any()) and not bool(r.dx[1, 3:].any()) and not bool(r.dg[1, 3:].any())


def test_lengths_outside_the_batch_are_clamped():
    c = inputs(2, 40, 8, "given", F32)
    L = torch.tensor([1000, -5], dtype=torch.int32, device="cuda")
    y, s = hla.gated_forward(c["x"], c["g"], state_in=c["state_in"], return_state=True, lengths=L)
    ry, rs, Ey, Es = ref.gated_forward(c["x"], c["g"], "given", None, c["state_in"], L.clamp(0, 40))
    ref.close(y, ry, Ey, "y")
    ref.close(s, rs, Es, "state_out")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chain_longer_than_one_look_back(dtype):
    """71 and more tiles of one chain: beyond the maps that one look-back keeps."""
    check(inputs(1, 128 * 71 + 5, 2, "given", dtype, seed=3))


@pytest.mark.parametrize("layout", ["packed", "time_major", "odd_offset", "odd_stride", "broadcast"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(layout, dtype):
    B, n, d = 3, 150, 48
    c = inputs(B, n, d, "sigmoid", dtype, seed=9)
    out = None
    if layout == "packed":       # x and g side by side in one projection, dx and dg too
        xg = torch.cat([c["x"], c["g"]], -1)
        c["x"], c["g"] = xg[..., :d], xg[..., d:]
        dxg = torch.zeros(B, n, 2 * d, dtype=dtype, device="cuda")
        out = dxg[..., :d], dxg[..., d:]
    elif layout == "time_major":
        c["x"], c["g"], c["dy"] = (c[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "g", "dy"))
        out = tuple(torch.zeros(n, B, d, dtype=dtype, device="cuda").transpose(0, 1) for _ in range(2))
    elif layout == "odd_offset":  # starts on an odd element
        for k in ("x", "g"):
            flat = torch.zeros(B * n * d + 1, dtype=dtype, device="cuda")
            flat[1:] = c[k].reshape(-1)
            c[k] = flat[1:].view(B, n, d)
    elif layout == "odd_stride":
        wide = torch.zeros(B, n, d + 1, dtype=dtype, device="cuda")
        wide[..., :d] = c["g"]
        c["g"] = wide[..., :d]
    else:                        # one gate for the batch
        c["g"] = c["g"][:1].expand(B, n, d)
    y = hla.gated_forward(c["x"], c["g"], "sigmoid", state_in=c["state_in"])
    ry, _, Ey, _ = ref.gated_forward(c["x"], c["g"], "sigmoid", None, c["state_in"])
    ref.close(y, ry, Ey, "y")
    r = hla.gated_backward(c["x"], c["g"], y, c["dy"], "sigmoid", state_in=c["state_in"], out=out)
    want = ref.gated_backward(c["x"], c["g"], y, c["dy"], "sigmoid", None, c["state_in"])
    for name in ("dx", "dg"):
        ref.close(getattr(r, name), *want[name], name)


@pytest.mark.parametrize("gate", GATES)
def test_resume_and_steps_continue_a_forward(gate):
    B, n, d = 2, 300, 66
    c = inputs(B, n, d, gate, BF16, seed=4)
    _, s = hla.gated_forward(c["x"][:, :170], c["g"][:, :170], gate, c["rate"], state_in=c["state_in"], return_state=True)
    y2, s = hla.gated_forward(c["x"][:, 170:295], c["g"][:, 170:295], gate, c["rate"], state_in=s, return_state=True)
    ry, rs, Ey, Es = ref.gated_forward(c["x"], c["g"], gate, c["rate"], c["state_in"])
    ref.close(y2, ry[:, 170:295], Ey[:, 170:295], "resumed y")
    for t in range(295, n):
        y, s2 = hla.gated_step(s, c["x"][:, t], c["g"][:, t], gate, c["rate"])
        assert s2 is s
        ref.close(y, ry[:, t], Ey[:, t], f"step {t}")
    ref.close(s, rs, Es, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [1, 37, 64])
def test_step_with_idle_sequences_and_a_second_state(dtype, d):
    c = inputs(4, 1, d, "rate", dtype, seed=2)
    L = torch.tensor([1, 0, 5, -1], dtype=torch.int32, device="cuda")
    state, nxt = c["state_in"].clone(), torch.full_like(c["state_in"], 7.0)
    out = torch.full((4, d), 7.0, dtype=dtype, device="cuda")
    hla.gated_step(state, c["x"][:, 0], c["g"][:, 0], "rate", c["rate"], lengths=L, state_out=nxt, out=out)
    assert torch.equal(state, c["state_in"])
    ry, rs, Ey, Es = ref.gated_forward(c["x"], c["g"], "rate", c["rate"], c["state_in"])
    for b in (0, 2):
        ref.close(out[b], ry[b, 0], Ey[b, 0], "y")
        ref.close(nxt[b], rs[b], Es[b], "state")
    for b in (1, 3):
        assert bool((out[b] == 7).all()) and bool((nxt[b] == 7).all())


@pytest.mark.parametrize("n", [0])
def test_no_tokens(n):
    c = inputs(2, 1, 5, "rate", F32)
    e = c["x"][:, :0]
    y, s = hla.gated_forward(e, e, "rate", c["rate"], state_in=c["state_in"], return_state=True)
    assert y.shape == (2, 0, 5) and torch.equal(s, c["state_in"])
    r = hla.gated_backward(e, e, e, e, "rate", c["rate"], d_state_out=c["d_state"], want_dstate=True)
    assert torch.equal(r.d_state_in, c["d_state"]) and not bool(r.d_rate.any())


def test_gates_at_their_ends():
    """Gates that are exactly 0 or 1, logits far out, an infinite input."""
    inf = float("inf")
    z = torch.tensor([-inf, -200.0, -90.0, -30.0, 0.0, 30.0, 90.0, inf], device="cuda")
    x = torch.ones(1, 3, 8, device="cuda")
    g = z.expand(1, 3, 8).contiguous()
    for gate, rate in (("sigmoid", None), ("rate", torch.ones(8, device="cuda"))):
        y = hla.gated_forward(x, g, gate, rate)
        ry, _, Ey, _ = ref.gated_forward(x, g, gate, rate)
        # sigma under the smallest normal float comes out as zero
        ref.close(y, ry, Ey + 1e-18, gate)
        r = hla.gated_backward(x, g, y, torch.ones_like(y), gate, rate)
        assert all(bool(torch.isfinite(t).all()) for t in (r.dx, r.dg))
    g01 = torch.tensor([0.0, 1.0], device="cuda").expand(1, 3, 2).contiguous()
    y = hla.gated_forward(x[..., :2].contiguous(), g01)
    assert y[0].tolist() == [[1.0, 1.0], [1.0, 2.0], [1.0, 3.0]]
    x[0, 1, 0] = inf
    y = hla.gated_forward(x, torch.full_like(x, 0.5))
    assert torch.isinf(y[0, 1:, 0]).all() and torch.isfinite(y[0, :, 1:]).all()


@pytest.mark.parametrize("gate", GATES)
def test_gradient_against_differences(gate):
    """Directional differences of the kernel's own forward in fp32: with step e the
    difference is off by e^2 / 6 times a third derivative and by rounding over e."""
    B, n, d = 1, 6, 4
    c = inputs(B, n, d, gate, F32, seed=8)
    w = c["dy"].double()
    names = ["x", "g", "state_in"] + (["rate"] if gate == "rate" else [])
    gen = torch.Generator(device="cuda").manual_seed(1)
    dirs = {k: torch.randn(c[k].shape, generator=gen, device="cuda") * (0.25 if k == "rate" else 1) for k in names}

    def loss(e):
        a = {k: c[k] + e * dirs[k] if k in dirs else c[k] for k in ("x", "g", "state_in", "rate")}
        y, s = hla.gated_forward(a["x"], a["g"], gate, a["rate"], state_in=a["state_in"], return_state=True)
        return float((y.double() * w).sum() + (s.double() * c["d_state"].double()).sum())

    y = hla.gated_forward(c["x"], c["g"], gate, c["rate"], state_in=c["state_in"])
    r = hla.gated_backward(c["x"], c["g"], y, c["dy"], gate, c["rate"], state_in=c["state_in"],
                           d_state_out=c["d_state"], want_dstate=True)
    got = {"x": r.dx, "g": r.dg, "state_in": r.d_state_in, "rate": r.d_rate}
    slope = sum(float((got[k].double() * dirs[k].double()).sum()) for k in names)
    e = 2.0 ** -9
    diff = (loss(e) - loss(-e)) / (2 * e)
    half = (loss(2 * e) - loss(-2 * e)) / (4 * e)  # e^2 terms: half - diff = 3 (diff - slope)
    noise = 64 * 2.0 ** -24 * (float(w.abs().sum()) + 10) / e
    assert abs(diff - slope) <= abs(half - diff) + noise, (diff, half, slope)


def test_same_bits_on_every_call():
    c = inputs(2, 3000, 64, "rate", BF16, seed=6)
    ws = hla.gated_workspace(c["x"])
    first = None
    for _ in range(5):
        y, s = hla.gated_forward(c["x"], c["g"], "rate", c["rate"], return_state=True, workspace=ws)
        r = hla.gated_backward(c["x"], c["g"], y, c["dy"], "rate", c["rate"], want_dstate=True, workspace=ws)
        now = (y, s, r.dx, r.dg, r.d_rate, r.d_state_in)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_one_workspace_for_calls_of_different_sizes():
    big, small = inputs(3, 900, 130, "rate", BF16, seed=1), inputs(2, 333, 65, "sigmoid", F32, seed=2)
    ws = hla.gated_workspace(big["x"])
    for _ in range(3):
        check(big, workspace=ws)
        check(small, workspace=ws)


def test_captured_calls_on_a_shared_workspace():
    """Two graphs whose calls use one workspace, replayed in turn on new inputs."""
    cs = [inputs(2, 700, 64, "rate", BF16, seed=1), inputs(1, 1300, 32, "sigmoid", BF16, seed=2)]
    ws = hla.gated_workspace(torch.empty(2, 1300, 64, dtype=BF16, device="cuda"))
    graphs, outs = [], []
    for c in cs:
        def call():
            y, s = hla.gated_forward(c["x"], c["g"], c["gate"], c["rate"], state_in=c["state_in"], return_state=True,
                                     workspace=ws)
            r = hla.gated_backward(c["x"], c["g"], y, c["dy"], c["gate"], c["rate"], state_in=c["state_in"],
                                   d_state_out=c["d_state"], want_dstate=True, workspace=ws)
            return y, s, r
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call()
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for k in range(3):
        for c, g in zip(cs, graphs):
            c["x"].copy_(torch.randn_like(c["x"], dtype=F32).to(BF16))
            g.replay()
    torch.cuda.synchronize()
    hla.hla_sync_status()
    for c, (y, s, r) in zip(cs, outs):
        ry, rs, Ey, Es = ref.gated_forward(c["x"], c["g"], c["gate"], c["rate"], c["state_in"])
        ref.close(y, ry, Ey, "y")
        ref.close(s, rs, Es, "state")
        want = ref.gated_backward(c["x"], c["g"], y, c["dy"], c["gate"], c["rate"], c["state_in"], c["d_state"])
        for name, (val, bound) in want.items():
            ref.close(getattr(r, name), val, bound, name)


def test_calls_on_another_stream():
    c = inputs(2, 400, 64, "sigmoid", BF16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = hla.gated_forward(c["x"], c["g"], "sigmoid", stream=st)
    z = hla.gated_forward(c["x"], c["g"], "sigmoid", stream=st.cuda_stream)
    st.synchronize()
    ry, _, Ey, _ = ref.gated_forward(c["x"], c["g"], "sigmoid")
    ref.close(y, ry, Ey, "y")
    assert torch.equal(y, z)


def test_offsets_beyond_32_bits():
    """A token stride that takes the last rows beyond 2^32 elements."""
    st, n, d = 1 << 28, 20, 8
    buf = torch.empty(n * st, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (1, n, d), (0, st, 1))
    c = inputs(1, n, d, "given", BF16)
    x.copy_(c["x"])
    y = hla.gated_forward(x, c["g"], "given")
    ry, _, Ey, _ = ref.gated_forward(c["x"], c["g"], "given")
    ref.close(y, ry, Ey, "y")


def test_wrapper_refusals():
    c = inputs(2, 10, 8, "given", BF16)
    with pytest.raises(ValueError, match="gate"):
        hla.gated_forward(c["x"], c["g"], "other")
    with pytest.raises(ValueError, match="rate"):
        hla.gated_forward(c["x"], c["g"], "rate")
    with pytest.raises(ValueError, match="rate"):
        hla.gated_forward(c["x"], c["g"], "given", rate=torch.ones(8, device="cuda"))
    with pytest.raises(TypeError):
        hla.gated_forward(c["x"], c["g"].float())
    with pytest.raises(TypeError):
        hla.gated_forward(c["x"].half(), c["g"].half())
    with pytest.raises(ValueError, match="shape"):
        hla.gated_forward(c["x"], c["g"][:, :5])
    with pytest.raises(ValueError, match="adjacent"):
        hla.gated_forward(c["x"], torch.empty(2, 8, 10, dtype=BF16, device="cuda").transpose(1, 2))
    with pytest.raises(ValueError):
        hla.gated_forward(c["x"], c["g"], lengths=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        hla.gated_forward(c["x"], c["g"], lengths=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(hla.HlaError, match="overlap"):
        hla.gated_forward(c["x"], c["g"], out=torch.empty(1, 10, 8, dtype=BF16, device="cuda").expand(2, 10, 8))
    with pytest.raises(hla.HlaError, match="may not be"):
        hla.gated_forward(c["x"], c["g"], out=c["x"])
    x = torch.zeros(1, 300, 8, dtype=BF16, device="cuda")
    with pytest.raises(hla.HlaError, match="workspace too small"):
        hla.gated_forward(x, x, workspace=hla.new_workspace(256))
    with pytest.raises(ValueError):
        hla.gated_forward(c["x"].cpu(), c["g"].cpu())


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,n,d,ragged", [(40, 1, 66, False), (2, 700, 1280, False), (13, 1500, 214, True), (3, 383, 1000, True),
                                          (1, 769, 2600, False)])
def test_many_channels(B, n, d, ragged, gate, dtype):
    """Enough channels that each CTA walks its sequence from end to end."""
    c = inputs(B, n, d, gate, dtype, seed=n)
    L = None
    if ragged:
        L = torch.tensor([n, 0, 1, n - 1, n // 2, 255, 256, 257, 384, 5, n, 100, 3][:B], dtype=torch.int32, device="cuda").clamp(max=n)
    y, s, r = check(c, lengths=L)
    if ragged:  # nothing is written behind the lengths
        dead = (torch.arange(n, device="cuda")[None, :, None] >= L[:, None, None]).expand_as(y)
        mark = torch.full_like(y, 7.0)
        hla.gated_forward(c["x"], c["g"], gate, c["rate"], lengths=L, out=mark)
        o = torch.full_like(y, 7.0), torch.full_like(y, 7.0)
        hla.gated_backward(c["x"], c["g"], y, c["dy"], gate, c["rate"], lengths=L, out=o)
        assert all(bool((t[dead] == 7).all()) for t in (mark,) + o)


def test_offsets_beyond_32_bits_with_many_channels():
    st, n, d = 1 << 28, 20, 2560
    buf = torch.empty((n - 1) * st + d, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (1, n, d), (0, st, 1))
    c = inputs(1, n, d, "sigmoid", BF16)
    x.copy_(c["x"])
    y = hla.gated_forward(x, c["g"], "sigmoid")
    ry, _, Ey, _ = ref.gated_forward(c["x"], c["g"], "sigmoid")
    ref.close(y, ry, Ey, "y")
    r = hla.gated_backward(x, c["g"], y, c["dy"], "sigmoid")
    want = ref.gated_backward(c["x"], c["g"], y, c["dy"], "sigmoid")
    ref.close(r.dg, *want["dg"], "dg")


@pytest.mark.parametrize("st", [5_590_000, 5_600_000])
def test_many_channels_with_tokens_far_apart(st):
    """Token strides on both sides of the largest whose offsets within a tile have 32 bits."""
    n, d = 390, 2560  # more than a tile of tokens
    c = inputs(1, n, d, "sigmoid", BF16, seed=4)
    far = torch.empty((n - 1) * st + d, dtype=BF16, device="cuda").as_strided((1, n, d), (0, st, 1))
    for name in ("x", "g", "dy"):
        far.copy_(c[name])
        check(dict(c, **{name: far}))
    y = hla.gated_forward(c["x"], c["g"], "sigmoid", state_in=c["state_in"])
    assert torch.equal(hla.gated_forward(c["x"], c["g"], "sigmoid", state_in=c["state_in"], out=far), far)
    assert float((far.float() - y.float()).abs().max()) <= 2 ** -7 * float(y.float().abs().max())
