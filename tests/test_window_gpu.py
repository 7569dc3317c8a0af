"""Windowed attention with first tokens that stay visible (hla_window_forward, _backward,
_step, _cache_fill) against its 64-bit form."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import constant_state_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def inputs(B, H, Hkv, n, nk, d, dv, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    return r(B, H, n, d), r(B, Hkv, nk, d), r(B, Hkv, nk, dv), r(B, H, n, dv)


def rounded(dtype):
    """Half a step of what the tensor-core path rounds P and dS to (the CUDA-core path keeps them in fp32)."""
    return ref.half_step(BF16) if dtype == BF16 else 0.0


def check(q, k, v, do, window, sinks, lengths=None, scale=None, outs=None):
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    n, nk, dt = q.shape[2], k.shape[2], q.dtype
    o, lse = hla.window_forward(q, k, v, window, sinks, scale=scale, lengths=lengths, return_lse=True)
    hla.hla_sync_status()
    ro, rl, Eo, El = ref.window_forward(q, k, v, window, sinks, sc, lengths, rounded(dt))
    ref.close(o, ro, Eo, "o")
    ref.close(lse, rl, El, "lse")
    dq, dk, dv = hla.window_backward(q, k, v, o, lse, do, window, sinks, scale=scale, lengths=lengths, out=outs)
    hla.hla_sync_status()
    want = ref.window_backward(q, k, v, o, lse, do, window, sinks, sc, lengths, rounded(dt))
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.close(got, *want[name], name)
    return o, lse, dq, dk, dv


SHAPES = [
    # B, H, Hkv, n, nk, d, dv, window, sinks
    (1, 1, 1, 1, 1, 64, 64, 1, 0),
    (2, 2, 1, 5, 5, 16, 16, 3, 1),
    (1, 2, 2, 63, 63, 64, 64, 16, 4),
    (1, 4, 2, 64, 64, 32, 48, 64, 0),
    (2, 3, 1, 129, 129, 128, 128, 40, 7),
    (1, 2, 1, 200, 200, 80, 64, 1, 3),       # window of one: itself and the first tokens
    (1, 2, 2, 300, 300, 64, 128, 1000, 0),   # plain causal
    (1, 6, 2, 257, 257, 128, 128, 130, 130), # first tokens in two tiles
    (1, 1, 1, 150, 150, 64, 64, 20, 400),    # every token is a first token
    (1, 2, 1, 70, 333, 64, 64, 100, 4),      # continues 263 held keys
    (1, 8, 1, 1, 500, 128, 128, 128, 16),    # one query on held keys
    (1, 4, 4, 640, 640, 64, 64, 128, 1),     # window and tiles coincide
    (1, 1, 1, 1200, 1200, 32, 32, 33, 5),    # far shares of the first tokens
    (1, 2, 1, 130, 130, 40, 24, 64, 2),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,Hkv,n,nk,d,dv,window,sinks", SHAPES)
def test_forward_and_gradients(B, H, Hkv, n, nk, d, dv, window, sinks, dtype):
    check(*inputs(B, H, Hkv, n, nk, d, dv, dtype, seed=n + d), window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,dv", [(1, 1), (33, 17), (127, 65), (64, 20)])
def test_odd_widths(d, dv, dtype):
    check(*inputs(1, 2, 1, 140, 140, d, dv, dtype, seed=d), 50, 3)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 256])
@pytest.mark.parametrize("sinks", [0, 2, 64, 129])
def test_windows_around_the_tiles(window, sinks):
    check(*inputs(1, 2, 1, 321, 321, 64, 64, BF16, seed=window), window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(5, 2 ** 31 - 1), (2 ** 31 - 1, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_largest_window_and_sinks(window, sinks, dtype):
    check(*inputs(1, 2, 1, 300, 300, 64, 64, dtype, seed=9), window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,nk", [(260, 260), (100, 260)])
def test_padded_batch(n, nk, dtype):
    """Rows behind a length hold NaN and infinities, and outputs there stay as they were."""
    B, H, Hkv, d, W, S = 6, 4, 2, 64, 70, 5
    L = torch.tensor([260, 0, 1, 129, 259, 161], dtype=torch.int32, device="cuda")
    q, k, v, do = inputs(B, H, Hkv, n, nk, d, d, dtype, seed=3)
    deadk = (torch.arange(nk, device="cuda") >= L[:, None])[:, None, :, None]
    deadq = (torch.arange(nk - n, nk, device="cuda") >= L[:, None])[:, None, :, None]
    nan = torch.tensor(float("nan"), dtype=dtype, device="cuda")
    inf = torch.tensor(float("inf"), dtype=dtype, device="cuda")
    q, do = torch.where(deadq, nan, q), torch.where(deadq, inf, do)
    k, v = torch.where(deadk, inf, k), torch.where(deadk, nan, v)
    sc = d ** -0.5
    o = torch.full((B, H, n, d), 7.0, dtype=dtype, device="cuda")
    o, lse = hla.window_forward(q, k, v, W, S, lengths=L, return_lse=True, out=o)
    hla.hla_sync_status()
    assert bool((o[deadq.expand_as(o)] == 7).all())
    ro, rl, Eo, El = ref.window_forward(q, k, v, W, S, sc, L, rounded(dtype))
    ref.close(torch.where(deadq, torch.zeros_like(o), o), ro, Eo, "o")
    ref.close(lse, rl, El, "lse")
    on, ln = torch.where(deadq, nan, o), torch.where(deadq[..., 0], float("nan"), lse)
    outs = tuple(torch.full_like(t, 7.0) for t in (q, k, v))
    dq, dk, dv = hla.window_backward(q, k, v, on, ln, do, W, S, lengths=L, out=outs)
    hla.hla_sync_status()
    want = ref.window_backward(q, k, v, on, ln, do, W, S, sc, L, rounded(dtype))
    for name, got, dead in (("dq", dq, deadq), ("dk", dk, deadk), ("dv", dv, deadk)):
        assert bool((got[dead.expand_as(got)] == 7).all()), name
        ref.close(torch.where(dead, torch.zeros_like(got), got), *want[name], name)


def test_new_outputs_of_a_padded_batch_are_zero_behind_the_lengths():
    q, k, v, do = inputs(2, 2, 1, 150, 150, 64, 64, BF16)
    L = torch.tensor([150, 3], dtype=torch.int32, device="cuda")
    o, lse = hla.window_forward(q, k, v, 20, 1, lengths=L, return_lse=True)
    g = hla.window_backward(q, k, v, o, lse, do, 20, 1, lengths=L)
    assert not any(bool(t[1, :, 3:].any()) for t in (o, lse) + g)


@pytest.mark.parametrize("layout", ["tokens_first", "packed", "odd_offset", "odd_stride", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(layout, dtype):
    B, H, Hkv, n, d = 2, 4, 2, 200, 64
    q, k, v, do = inputs(B, H, Hkv, n, n, d, d, dtype, seed=5)
    outs = None
    if layout == "tokens_first":  # [B, n, H, d] as projections leave them
        q, k, v, do = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do))
        outs = tuple(torch.zeros_like(t) for t in (q, k, v))
        assert not outs[0].is_contiguous()
    elif layout == "packed":      # one projection's rows hold q, k and v, and their gradients
        pack = torch.cat([t.transpose(1, 2).reshape(B, n, -1) for t in (q, k, v)], -1)
        split = lambda p: tuple(x.unflatten(2, (-1, d)).transpose(1, 2) for x in p.split([H * d, Hkv * d, Hkv * d], -1))  # noqa: E731
        q, k, v = split(pack)
        outs = split(torch.zeros_like(pack))
    elif layout == "odd_offset":
        flat = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
        flat[1:] = q.reshape(-1)
        q = flat[1:].view(q.shape)
    elif layout == "odd_stride":
        wide = torch.zeros(B, Hkv, n, d + 1, dtype=dtype, device="cuda")
        wide[..., :d] = v
        v = wide[..., :d]
    else:                         # one key/value sequence for the batch
        k, v = k[:1].expand(B, Hkv, n, d), v[:1].expand(B, Hkv, n, d)
        outs = tuple(torch.zeros(B, h, n, d, dtype=dtype, device="cuda") for h in (H, Hkv, Hkv))
    check(q, k, v, do, 33, 2, outs=outs)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale, dtype):
    check(*inputs(1, 2, 1, 150, 150, 64, 64, dtype, seed=1), 60, 2, scale=scale)


def test_large_scores():
    """Scores in the hundreds, growing along the sequence: the running maximum moves at every tile."""
    q, k, v, do = inputs(1, 2, 1, 500, 500, 64, 64, F32, seed=2)
    k = k * torch.linspace(0.5, 20, 500, device="cuda")[:, None]
    check(q, k, v, do, 300, 4)
    check(q.to(BF16), k.to(BF16), v.to(BF16), do.to(BF16), 300, 4)
    check(q.to(BF16), k.flip(2).to(BF16), v.to(BF16), do.to(BF16), 300, 4)


def test_without_lse_and_same_bits():
    q, k, v, do = inputs(1, 4, 2, 700, 700, 64, 64, BF16, seed=2)
    o, lse = hla.window_forward(q, k, v, 100, 4, return_lse=True)
    assert torch.equal(o, hla.window_forward(q, k, v, 100, 4))
    first = hla.window_backward(q, k, v, o, lse, do, 100, 4)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, hla.window_backward(q, k, v, o, lse, do, 100, 4)))


def test_causality():
    """Later tokens do not reach earlier rows, nor tokens that have left the window."""
    q, k, v, _ = inputs(1, 2, 1, 400, 400, 64, 64, BF16, seed=2)
    o = hla.window_forward(q, k, v, 50, 3)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 200:], v2[:, :, 200:] = 3.0, -5.0
    assert torch.equal(o[:, :, :200], hla.window_forward(q, k2, v2, 50, 3)[:, :, :200])
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 3:100], v2[:, :, 3:100] = 3.0, -5.0
    assert torch.equal(o[:, :, 149:], hla.window_forward(q, k2, v2, 50, 3)[:, :, 149:])


def test_no_queries():
    q, k, v, _ = inputs(1, 2, 1, 4, 4, 64, 64, BF16)
    assert hla.window_forward(q[:, :, :0], k, v, 2).shape == (1, 2, 0, 64)


def test_gradient_against_differences():
    """Differences of the kernel's forward in fp32 along a random direction (the bound: the
    change of the difference when its step doubles, and rounding over the step)."""
    q, k, v, do = inputs(1, 2, 1, 20, 20, 8, 6, F32, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dirs = [torch.randn(t.shape, generator=gen, device="cuda") for t in (q, k, v)]

    def loss(e):
        o = hla.window_forward(*(t + e * x for t, x in zip((q, k, v), dirs)), 7, 2)
        return float((o.double() * do.double()).sum())

    o, lse = hla.window_forward(q, k, v, 7, 2, return_lse=True)
    g = hla.window_backward(q, k, v, o, lse, do, 7, 2)
    slope = sum(float((a.double() * b.double()).sum()) for a, b in zip(g, dirs))
    e = 2.0 ** -9
    diff, half = (loss(e) - loss(-e)) / (2 * e), (loss(2 * e) - loss(-2 * e)) / (4 * e)
    noise = 64 * 2.0 ** -24 * float(do.abs().sum()) / e
    assert abs(diff - slope) <= abs(half - diff) + noise, (diff, half, slope)


# ------------------------------------------------------------------ decoding
def step_ref(kc, vc, pos, q, k, v, window, sinks, scale, rnd):
    """o, its bound and the caches after the step, by the definition."""
    B, H, d = q.shape
    Hkv, G = k.shape[1], H // k.shape[1]
    kc, vc = kc.clone(), vc.clone()
    o, E = torch.zeros(B, H, v.shape[-1], dtype=torch.float64, device="cuda"), torch.zeros(B, H, v.shape[-1], dtype=torch.float64, device="cuda")
    for b in range(B):
        p = int(pos[b])
        if p < 0:
            continue
        at = p if p < sinks else sinks + (p - sinks) % window
        kc[b, :, at], vc[b, :, at] = k[b], v[b]
        m = min(p + 1, sinks + window)
        for h in range(H):
            kk, vv, qq = kc[b, h // G, :m].double(), vc[b, h // G, :m].double(), q[b, h].double()
            s = kk @ qq * scale
            delta = (d + 8) * ref.U * abs(scale) * (kk.abs() @ qq.abs())
            P = torch.softmax(s, 0)
            o[b, h] = P @ vv
            E[b, h] = (P * (2 * delta + 2 * delta.max() + 16 * ref.U + 2 * rnd + 2 * m * ref.U)) @ vv.abs()
    return o, E, kc, vc


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hkv,d,dv,window,sinks", [(2, 2, 64, 64, 1, 0), (4, 2, 128, 128, 100, 5), (8, 1, 64, 128, 300, 0),
                                                     (9, 1, 128, 64, 64, 64), (20, 1, 33, 17, 40, 3), (6, 2, 80, 40, 1000, 16),
                                                     (16, 1, 128, 128, 64, 0)])
def test_step(H, Hkv, d, dv, window, sinks, dtype):
    cap = sinks + window
    pos = torch.tensor([-1, 0, max(sinks - 1, 0), sinks, cap - 1, cap, 3 * cap + 7, (1 << 33) + 5, -9], device="cuda")
    B = pos.numel()
    gen = torch.Generator(device="cuda").manual_seed(H + d)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    q, k, v, kc, vc = r(B, H, d), r(B, Hkv, d), r(B, Hkv, dv), r(B, Hkv, cap, d), r(B, Hkv, cap, dv)
    unused = (torch.arange(cap, device="cuda") > pos[:, None])[:, None, :, None]
    kc, vc = kc.masked_fill(unused, float("nan")), vc.masked_fill(unused, float("inf"))
    out = torch.full((B, H, dv), 7.0, dtype=dtype, device="cuda")
    ro, E, rk, rv = step_ref(kc, vc, pos, q, k, v, window, sinks, d ** -0.5, rounded(dtype))
    o = hla.window_step(kc, vc, pos, q, k, v, window, sinks, out=out)
    hla.hla_sync_status()
    assert bool((o[0] == 7).all()) and bool((o[8] == 7).all())
    ref.close(o[1:8], ro[1:8], E[1:8], "o")
    for got, want in ((kc, rk), (vc, rv)):
        assert torch.equal(got.nan_to_num(nan=99.0), want.nan_to_num(nan=99.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_strides(dtype):
    """A cache of [B, slots, Hkv, d], q, k, v in one row, and rows that start on odd elements."""
    B, H, Hkv, d, W, S = 3, 4, 2, 64, 50, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    for odd in (0, 1):
        kc, vc = (r(B, W + S, Hkv, d + odd).transpose(1, 2)[..., :d] for _ in range(2))
        row = r(B, (H + 2 * Hkv) * d + odd)[:, odd:].unflatten(1, (-1, d))
        q, k, v = row[:, :H], row[:, H:H + Hkv], row[:, H + Hkv:]
        pos = torch.tensor([0, 30, 300], device="cuda")
        ro, E, rk, rv = step_ref(kc, vc, pos, q, k, v, W, S, d ** -0.5, rounded(dtype))
        o = hla.window_step(kc, vc, pos, q, k, v, W, S)
        ref.close(o, ro, E, "o")
        assert torch.equal(kc, rk) and torch.equal(vc, rv)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fill_then_steps_continue_a_forward(dtype):
    """A ragged prompt into the ring, then token by token, against one forward over all tokens."""
    B, H, Hkv, n, d, dv, W, S, more = 5, 4, 2, 210, 64, 40, 50, 6, 70
    q, k, v, _ = inputs(B, H, Hkv, n + more, n + more, d, dv, dtype, seed=6)
    L = torch.tensor([210, 0, 3, 56, 57], dtype=torch.int32, device="cuda")
    kc, vc = hla.window_cache(B, Hkv, W, S, d, dv, dtype)
    kc.fill_(float("nan")), vc.fill_(float("nan"))
    hla.window_cache_fill(kc, vc, k[:, :, :n], v[:, :, :n], W, S, lengths=L)
    ro, _, E, _ = ref.window_forward(q, k, v, W, S, d ** -0.5, None, rounded(dtype))
    pos = L.long()
    rows = torch.arange(B, device="cuda")
    for _ in range(more):
        o = hla.window_step(kc, vc, pos, q[rows, :, pos], k[rows, :, pos], v[rows, :, pos], W, S)
        ref.close(o, ro[rows, :, pos], E[rows, :, pos], "o")
        pos += 1
    hla.hla_sync_status()


def test_fill_leaves_other_slots():
    k = torch.randn(1, 1, 4, 8, device="cuda")
    kc, vc = torch.full((1, 1, 12, 8), 7.0, device="cuda"), torch.full((1, 1, 12, 8), 7.0, device="cuda")
    hla.window_cache_fill(kc, vc, k, k, 10, 2)
    assert torch.equal(kc[0, 0, :4], k[0, 0]) and bool((kc[0, 0, 4:] == 7).all())


def test_captured_calls_and_another_stream():
    q, k, v, do = inputs(2, 4, 2, 300, 300, 64, 64, BF16, seed=6)
    kc, vc = hla.window_cache(2, 2, 40, 2, 64)
    kc.zero_(), vc.zero_()
    pos = torch.tensor([5, 100], device="cuda")

    def call(stream=None):
        o, lse = hla.window_forward(q, k, v, 70, 3, return_lse=True, stream=stream)
        g = hla.window_backward(q, k, v, o, lse, do, 70, 3, stream=stream)
        s = hla.window_step(kc, vc, pos, q[:, :, 0], k[:, :, 0], v[:, :, 0], 40, 2, stream=stream)
        return (o, lse, s) + g

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(st)
    call(st.cuda_stream)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    q.copy_(torch.randn_like(q, dtype=F32).to(BF16))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))
    hla.hla_sync_status()


def test_wrapper_refusals():
    q, k, v, do = inputs(1, 4, 2, 10, 10, 16, 16, BF16)
    for kw, exc in ((dict(window=0), hla.HlaError), (dict(window=1 << 40), ValueError), (dict(window=4, sinks=-1), hla.HlaError),
                    (dict(window=4, scale=float("nan")), hla.HlaError)):
        with pytest.raises(exc):
            hla.window_forward(q, k, v, **kw)
    with pytest.raises(hla.HlaError):
        hla.window_forward(q[:, :3], k, v, 4)
    with pytest.raises(hla.HlaError):
        hla.window_forward(q, k[:, :, :5], v[:, :, :5], 4)  # fewer keys than queries
    with pytest.raises(ValueError):
        hla.window_forward(q, k, v[:, :, :5], 4)
    with pytest.raises(TypeError):
        hla.window_forward(q, k.float(), v, 4)
    with pytest.raises(hla.HlaError, match="may not be"):
        hla.window_forward(q, k, v, 4, out=q)
    with pytest.raises(hla.HlaError, match="overlap"):
        hla.window_forward(q, k, v, 4, out=torch.empty(1, 1, 10, 16, dtype=BF16, device="cuda").expand(1, 4, 10, 16))
    w = torch.zeros(1, 1, 4, 160, dtype=BF16, device="cuda")
    with pytest.raises(hla.HlaError) as e:
        hla.window_forward(w, w, w, 4)
    assert e.value.status == hla.HLA_ERR_UNSUPPORTED
    o, lse = hla.window_forward(q, k, v, 4, return_lse=True)
    with pytest.raises(hla.HlaError, match="workspace"):
        hla.window_backward(q, k, v, o, lse, do, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        hla.window_backward(q, k, v, o, lse.double(), do, 4)
    kc, vc = hla.window_cache(1, 2, 4, 1, 16)
    with pytest.raises(ValueError):
        hla.window_step(kc, vc, torch.zeros(1, dtype=torch.int64, device="cuda"), q[:, :, 0], k[:, :, 0], v[:, :, 0], 5, 1)
    with pytest.raises(TypeError):
        hla.window_step(kc, vc, torch.zeros(1, dtype=torch.int32, device="cuda"), q[:, :, 0], k[:, :, 0], v[:, :, 0], 4, 1)
