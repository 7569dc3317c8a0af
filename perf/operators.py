"""Workloads of the gated linear recurrence and of the windowed attention with first
tokens that stay visible: inputs, the plain form of each operator, its definition in
64 bits, and the bytes and operations it cannot do without.

Operators ("op" of a case):
  gated_forward, gated_backward, gated_step: h_t = a_t h_{t-1} + b_t over [B, n, d]
  window_forward, window_backward, window_step: softmax attention of a query at p over
      the keys j <= p with j > p - window or j < sinks
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
KINDS = ("given", "sigmoid", "rate")


# --------------------------------------------------------------------------- cases
def _gated(op, B, n, d, gate, dtype, ragged=False, name=None):
    c = {"op": op, "B": B, "n": n, "d": d, "gate": gate, "dtype": dtype, "ragged": ragged}
    return {"name": name, **c} if name else c


def _window(op, B, H, Hkv, n, d, window, sinks, dtype, ragged=False, name=None):
    c = {"op": op, "B": B, "H": H, "Hkv": Hkv, "n": n, "d": d, "window": window, "sinks": sinks, "dtype": dtype,
         "ragged": ragged}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of one stream through a scan layer: nothing but latency
        _gated("gated_step", 1, 1, 2048, "sigmoid", BF16, name="gated_step_b1_d2048"),
        # a serving batch of 256 streams, 32 heads of 128 channels each
        _gated("gated_step", 256, 1, 4096, "rate", BF16, name="gated_step_b256_d4096"),
        # padded batch of sequences of different lengths, an odd width, full precision
        _gated("gated_forward", 3, 5003, 1001, "given", F32, ragged=True, name="gated_fwd_ragged_f32_n5003_d1001"),
        # one long sequence (prefill or long-context training), 32 heads of 128 channels
        _gated("gated_forward", 1, 32768, 4096, "rate", BF16, name="gated_fwd_n32768_d4096"),
        # training step of a small layer, 8 heads of 64 channels
        _gated("gated_backward", 4, 2048, 512, "sigmoid", BF16, name="gated_bwd_b4_n2048_d512"),
        # training step of a wide layer, with the gradient of the learned rates
        _gated("gated_backward", 2, 8192, 4096, "rate", BF16, name="gated_bwd_b2_n8192_d4096"),
        # training or prefill at a short window, heads of 64, no shared key/value heads
        _window("window_forward", 4, 8, 8, 2048, 64, 256, 4, BF16, name="window_fwd_b4_h8_n2048_d64_w256"),
        # long prefill with shared key/value heads
        _window("window_forward", 1, 32, 8, 16384, 128, 2048, 16, BF16, name="window_fwd_h32_n16384_d128_w2048"),
        # training on a padded batch, odd lengths and window
        _window("window_backward", 3, 6, 2, 1501, 64, 301, 4, BF16, ragged=True, name="window_bwd_ragged_n1501_d64_w301"),
        # training step of a wide layer on long sequences
        _window("window_backward", 2, 16, 4, 8192, 128, 1024, 16, BF16, name="window_bwd_b2_h16_n8192_d128_w1024"),
        # one token of one stream over a full ring cache
        _window("window_step", 1, 32, 8, 1, 128, 4096, 16, BF16, name="window_step_b1_h32_d128_w4096"),
        # a serving batch of 64 streams at different positions, some still filling their rings
        _window("window_step", 64, 32, 8, 1, 128, 1024, 16, BF16, ragged=True, name="window_step_b64_h32_d128_w1024"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_forward", "gated_backward", "gated_step", "window_forward", "window_backward",
                     "window_step"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    ragged = rng.random() < 0.4
    if op.startswith("gated"):
        gate = rng.choice(KINDS)
        if op == "gated_step":
            return _gated(op, _log_int(rng, 1, 256), 1, _log_int(rng, 64, 4096), gate, dtype, ragged)
        while True:
            B, n, d = _log_int(rng, 1, 16), _log_int(rng, 1, 32768), _log_int(rng, 33, 4096)
            if rng.random() < 0.5:
                d = (d + 63) // 64 * 64
            if B * n * d * (2 if dtype == F32 else 1) <= 1 << 26:
                return _gated(op, B, n, d, gate, dtype, ragged)
    d = rng.choice([32, 64, 64, 80, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4])
    sinks = rng.choice([0, 1, 4, 16, 64])
    if op == "window_step":
        return _window(op, _log_int(rng, 1, 64), H, Hkv, 1, d, _log_int(rng, 16, 4096), sinks, dtype, ragged)
    while True:
        B, n, window = _log_int(rng, 1, 8), _log_int(rng, 1, 16384), _log_int(rng, 16, 4096)
        products = (4 if op == "window_forward" else 10) * B * H * n * (min(window, n) + sinks) * d
        # full precision does its products at the rate of fp32 arithmetic
        if products <= (5e11 if dtype == BF16 else 5e10):
            return _window(op, B, H, Hkv, n, d, window, sinks, dtype, ragged)


# --------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _lengths(case, gen, n):
    """Valid tokens of each sequence: the first is whole, the others anywhere from a few to all."""
    if not case["ragged"]:
        return None
    B = case["B"]
    u = torch.rand(B, generator=gen, device="cuda")
    L = (n * (0.05 + 0.95 * u)).long().clamp(1, n)
    L[0] = n
    return L.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    dt = _dt(case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": dict(case)}
    if case["op"].startswith("gated"):
        B, n, d = case["B"], case["n"], case["d"]
        shape = (B, d) if case["op"] == "gated_step" else (B, n, d)
        s["x"] = randn(*shape).to(dt)
        # gates that keep 1 to 1000 tokens, as trained ones do
        z = randn(*shape) + torch.linspace(0.0, 4.0, d, device="cuda")
        s["g"] = (torch.sigmoid(z) if case["gate"] == "given" else z).to(dt)
        del z
        s["rate"] = torch.exp(torch.linspace(math.log(0.01), math.log(2.0), d, device="cuda")) if case["gate"] == "rate" else None
        s["state"] = randn(B, d)
        if case["op"] == "gated_step":
            s["next"] = torch.zeros_like(s["state"])
            # a ragged serving batch has idle slots
            s["lengths"] = (torch.rand(B, generator=gen, device="cuda") < 0.8).to(torch.int32) if case["ragged"] else None
            s["y"] = torch.zeros_like(s["x"])
            if case["ragged"]:
                s["next"].copy_(s["state"])
            return s
        s["lengths"] = _lengths(case, gen, n)
        if case["op"] == "gated_backward":
            s["y"] = _gated_forward(s)[0]
            s["dy"] = randn(*shape).to(dt)
            s["dstate"] = randn(B, d)
        return s
    B, H, Hkv, n, d = case["B"], case["H"], case["Hkv"], case["n"], case["d"]
    if case["op"] == "window_step":
        slots = case["window"] + case["sinks"]
        s["q"] = randn(B, H, d).to(dt)
        s["k"], s["v"] = randn(B, Hkv, d).to(dt), randn(B, Hkv, d).to(dt)
        s["kc"], s["vc"] = randn(B, Hkv, slots, d).to(dt), randn(B, Hkv, slots, d).to(dt)
        pos = torch.full((B,), 3 * slots + 5, device="cuda", dtype=torch.int64)
        if case["ragged"]:  # from an empty cache to several times round the ring; now and then an idle slot
            u = torch.rand(B, generator=gen, device="cuda")
            pos = (u * 4 * slots).long() - slots // 16
        s["pos"] = pos
        s["o"] = torch.zeros(B, H, d, device="cuda", dtype=dt)
        return s
    s["q"] = randn(B, H, n, d).to(dt)
    s["k"], s["v"] = randn(B, Hkv, n, d).to(dt), randn(B, Hkv, n, d).to(dt)
    s["lengths"] = _lengths(case, gen, n)
    if case["op"] == "window_backward":
        s["o"], s["lse"] = _window_forward(s)
        s["do"] = randn(B, H, n, d).to(dt)
    return s


# --------------------------------------------------------------------------- plain forms: gated
def _gates(case, g, rate):
    """a_t and the factor of x_t, in 32 bits."""
    g = g.float()
    if case["gate"] == "given":
        return g, torch.ones((), device=g.device)
    if case["gate"] == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(-g)
    u = rate * torch.sigmoid(g)
    return torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def _scan(a, b):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... along dim 1, by doubling."""
    n, k = a.shape[1], 1
    while k < n:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _valid(s, n):
    """[B, n, 1]: token t is below its sequence's length."""
    if s["lengths"] is None:
        return None
    return (torch.arange(n, device="cuda") < s["lengths"][:, None])[..., None]


def _gated_forward(s):
    x = s["x"]
    a, f = _gates(s["case"], s["g"], s["rate"])
    b = f * x.float()
    ok = _valid(s, x.shape[1])
    if ok is not None:
        a, b = torch.where(ok, a, 1.0), torch.where(ok, b, 0.0)
    b = torch.cat([b[:, :1] + a[:, :1] * s["state"][:, None], b[:, 1:]], 1)
    h = _scan(a, b)
    state = h[:, -1].contiguous()
    y = h if ok is None else torch.where(ok, h, 0.0)
    return y.to(x.dtype), state


def _gated_backward(s):
    case, dt = s["case"], s["x"].dtype
    x, dy = s["x"].float(), s["dy"].float()
    a, f = _gates(case, s["g"], s["rate"])
    ok = _valid(s, x.shape[1])
    if ok is not None:
        a, dy = torch.where(ok, a, 1.0), torch.where(ok, dy, 0.0)
    c = a * dy
    c = torch.cat([c[:, :-1], c[:, -1:] + a[:, -1:] * s["dstate"][:, None]], 1)
    c = _scan(a.flip(1), c.flip(1)).flip(1)
    gh = dy + torch.cat([c[:, 1:], s["dstate"][:, None]], 1)
    before = torch.cat([s["state"][:, None], s["y"][:, :-1].float()], 1)
    drate = None
    dx = gh * f
    if case["gate"] == "given":
        dg = gh * before
    elif case["gate"] == "sigmoid":
        dg = gh * (before - x) * (a * f)
    else:
        sg = torch.sigmoid(s["g"].float())
        du = gh * (torch.where(f > 0, a * a / f, 0.0) * x - a * before)
        dg = du * s["rate"] * sg * (1 - sg)
        dr = du * sg
        drate = (dr if ok is None else torch.where(ok, dr, 0.0)).sum((0, 1))
    if ok is not None:
        dx, dg = torch.where(ok, dx, 0.0), torch.where(ok, dg, 0.0)
    return (dx.to(dt), dg.to(dt), c[:, 0].contiguous()) + (() if drate is None else (drate,))


def _gated_step(s):
    a, f = _gates(s["case"], s["g"], s["rate"])
    h = a * s["state"] + f * s["x"].float()
    y = h.to(s["x"].dtype)
    if s["lengths"] is not None:
        live = s["lengths"][:, None] > 0
        h, y = torch.where(live, h, s["next"]), torch.where(live, y, s["y"])
    return y, h


# --------------------------------------------------------------------------- plain forms: window
BLOCK = 256  # queries that share one gathered band of keys


def _bands(s):
    """Queries in blocks against the band of keys each block can see, and against the first
    tokens.  Returns the block size, the keys' indices [blocks, span], and what of the band
    [B, blocks, rows, span] and of the first tokens [B, blocks, rows, sinks] is visible."""
    case = s["case"]
    n, S = case["n"], min(case["sinks"], case["n"])
    W = min(case["window"], n)
    c = min(BLOCK, n)
    nb = -(-n // c)
    dev = s["q"].device
    p = (torch.arange(nb, device=dev) * c)[:, None] + torch.arange(c, device=dev)  # [nb, c]
    j = (torch.arange(nb, device=dev) * c)[:, None] - (W - 1) + torch.arange(W - 1 + c, device=dev)  # [nb, span]
    L = s["lengths"].long() if s["lengths"] is not None else torch.full((case["B"],), n, device=dev)
    band = (j[:, None] <= p[..., None]) & (j[:, None] > p[..., None] - W) & (j[:, None] >= S)
    live = (p[None] < L[:, None, None])[..., None]  # [B, nb, c, 1]
    first = torch.arange(S, device=dev) <= p[..., None]
    return c, nb, j.clamp(0, n - 1), band[None] & live, first[None] & live


def _blocks(x, Hkv, c, nb):
    """[B, H, n, d] to [B, Hkv, blocks, group * c, d]: the rows that share a band of keys."""
    B, H, n, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * c - n))
    return x.view(B, Hkv, H // Hkv, nb, c, d).transpose(2, 3).reshape(B, Hkv, nb, H // Hkv * c, d)


def _unblock(x, H, n):
    """The inverse of _blocks."""
    B, Hkv, nb, gc, d = x.shape
    G = H // Hkv
    return x.view(B, Hkv, nb, G, gc // G, d).transpose(2, 3).reshape(B, H, -1, d)[:, :, :n]


def _scores(s):
    case = s["case"]
    c, nb, j, band, first = _bands(s)
    G = case["H"] // case["Hkv"]
    q = _blocks(s["q"], case["Hkv"], c, nb)
    k, v = s["k"].float(), s["v"].float()
    S = first.shape[-1]
    sees = torch.cat([first, band], -1)  # [B, nb, c, S + span]
    sees = sees[:, None, :, None].expand(-1, 1, -1, G, -1, -1).reshape(sees.shape[0], 1, nb, G * c, -1)
    kb, vb = k[:, :, j], v[:, :, j]
    sc = torch.cat([q @ k[:, :, None, :S].transpose(-1, -2), q @ kb.transpose(-1, -2)], -1) / math.sqrt(case["d"])
    return c, nb, j, S, q, k, v, kb, vb, sc.masked_fill_(~sees, -math.inf), sees


def _window_forward(s):
    case, dt = s["case"], s["q"].dtype
    c, nb, j, S, q, k, v, kb, vb, sc, sees = _scores(s)
    live = sees.any(-1, keepdim=True)
    m = torch.where(live, sc.amax(-1, keepdim=True), 0.0)
    e = torch.exp(sc - m)
    l = e.sum(-1, keepdim=True)
    o = (e[..., :S] @ v[:, :, None, :S] + e[..., S:] @ vb) / torch.where(live, l, 1.0)
    lse = torch.where(live, m + torch.log(l), 0.0)
    return _unblock(o, case["H"], case["n"]).to(dt), _unblock(lse, case["H"], case["n"])[..., 0].contiguous()


def _window_backward(s):
    case, dt = s["case"], s["q"].dtype
    H, Hkv, n = case["H"], case["Hkv"], case["n"]
    c, nb, j, S, q, k, v, kb, vb, sc, sees = _scores(s)
    do = _blocks(s["do"], Hkv, c, nb)
    o = _blocks(s["o"], Hkv, c, nb)
    lse = _blocks(s["lse"][..., None], Hkv, c, nb)
    P = torch.where(sees, torch.exp(sc - lse), 0.0)
    do = torch.where(sees.any(-1, keepdim=True), do, 0.0)
    del sc
    dP = torch.cat([do @ v[:, :, None, :S].transpose(-1, -2), do @ vb.transpose(-1, -2)], -1)
    dS = P * (dP - (do * o).sum(-1, keepdim=True)) / math.sqrt(case["d"])
    del dP
    dq = _unblock(dS[..., :S] @ k[:, :, None, :S] + dS[..., S:] @ kb, H, n)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    dk.index_add_(2, j.reshape(-1), (dS[..., S:].transpose(-1, -2) @ q).flatten(2, 3))
    dv.index_add_(2, j.reshape(-1), (P[..., S:].transpose(-1, -2) @ do).flatten(2, 3))
    dk[:, :, :S] += (dS[..., :S].transpose(-1, -2) @ q).sum(2)
    dv[:, :, :S] += (P[..., :S].transpose(-1, -2) @ do).sum(2)
    return dq.to(dt), dk.to(dt), dv.to(dt)


def _window_step(s):
    case = s["case"]
    B, H, Hkv, d, W, S = (case[x] for x in ("B", "H", "Hkv", "d", "window", "sinks"))
    pos, kc, vc = s["pos"], s["kc"], s["vc"]
    live = pos >= 0
    slot = torch.where(pos < S, pos, S + (pos - S) % W).clamp(min=0)
    at = torch.arange(B, device=pos.device)
    kc[at, :, slot] = torch.where(live[:, None, None], s["k"], kc[at, :, slot])
    vc[at, :, slot] = torch.where(live[:, None, None], s["v"], vc[at, :, slot])
    q = s["q"].float().view(B, Hkv, H // Hkv, d)
    sc = q @ kc.float().transpose(-1, -2) / math.sqrt(d)
    sees = (torch.arange(S + W, device=pos.device) <= pos[:, None])[:, None, None]
    sc = sc.masked_fill(~sees, -math.inf)
    m = torch.where(live[:, None, None, None], sc.amax(-1, keepdim=True), 0.0)
    e = torch.exp(sc - m)
    o = (e @ vc.float()) / torch.where(live[:, None, None, None], e.sum(-1, keepdim=True), 1.0)
    o = torch.where(live[:, None, None], o.view(B, H, d).to(s["o"].dtype), s["o"])
    return o, kc, vc


# --------------------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "gated_forward":
            return _gated_forward(s)
        if op == "gated_backward":
            return _gated_backward(s)
        if op == "gated_step":
            return _gated_step(s)
        if op == "window_forward":
            return _window_forward(s)
        if op == "window_backward":
            return _window_backward(s)
        return _window_step(s)
    import causal_prefix_scan_gb300 as hla
    if op in ("gated_forward", "gated_backward") and "ws" not in s:  # kept by the program from its first call on
        s["ws"] = hla.gated_workspace(s["x"])
    if op == "gated_forward":
        return hla.gated_forward(s["x"], s["g"], gate=case["gate"], rate=s["rate"], state_in=s["state"],
                                 return_state=True, lengths=s["lengths"], workspace=s["ws"])
    if op == "gated_backward":
        r = hla.gated_backward(s["x"], s["g"], s["y"], s["dy"], gate=case["gate"], rate=s["rate"], state_in=s["state"],
                               d_state_out=s["dstate"], want_dstate=True, lengths=s["lengths"], workspace=s["ws"])
        return (r.dx, r.dg, r.d_state_in) + (() if r.d_rate is None else (r.d_rate,))
    if op == "gated_step":
        return hla.gated_step(s["state"], s["x"], s["g"], gate=case["gate"], rate=s["rate"], lengths=s["lengths"],
                              state_out=s["next"], out=s["y"])
    W, S = case["window"], case["sinks"]
    if op == "window_forward":
        return hla.window_forward(s["q"], s["k"], s["v"], W, sinks=S, lengths=s["lengths"], return_lse=True)
    if op == "window_backward":
        if "ws" not in s:
            s["ws"] = hla.window_workspace(s["q"], s["k"], s["v"], W, sinks=S)
        return hla.window_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], W, sinks=S, lengths=s["lengths"],
                                   workspace=s["ws"])
    o = hla.window_step(s["kc"], s["vc"], s["pos"], s["q"], s["k"], s["v"], W, sinks=S, out=s["o"])
    return o, s["kc"], s["vc"]


# --------------------------------------------------------------------------- floors
def _pairs(n, W, S):
    """Visible (query, key) pairs of one head over n tokens."""
    band = sum_to(min(n, W)) + max(0, n - W) * W
    first = 0  # first tokens that have left the window: query p misses min(S, p - W + 1) of them
    if n > W:
        m = n - W
        k = min(m, S)
        first = sum_to(k) + (m - k) * S
    return band + first


def sum_to(k):
    return k * (k + 1) // 2


def work(case):
    e = 4 if case["dtype"] == F32 else 2
    B, n, d, op = case["B"], case["n"], case["d"], case["op"]
    if op == "gated_step":
        live = 0.8 * B if case["ragged"] else B
        return {"bytes": live * d * (3 * e + 8) + (4 * d if case["gate"] == "rate" else 0), "flops": 6 * live * d}
    # expected lengths of the sequences of a padded batch: the first is whole, the others 5 % to all of it
    each = [n * (0.05 + 0.95 * (i + 0.5) / 16) for i in range(16)] if case["ragged"] else [n]
    mean = lambda f: f(n) + (B - 1) * sum(f(max(1, int(x))) for x in each) / len(each)  # noqa: E731
    tokens = mean(lambda x: x)
    if op.startswith("gated"):
        N, st = tokens * d, 4 * B * d
        rate = 4 * d if case["gate"] == "rate" else 0
        if op == "gated_backward":
            streams = 5 if case["gate"] == "given" else 6
            return {"bytes": streams * N * e + 3 * st + 2 * rate, "flops": 12 * N}
        return {"bytes": 3 * N * e + 2 * st + rate, "flops": 6 * N}
    H, Hkv, W, S = case["H"], case["Hkv"], case["window"], case["sinks"]
    if op == "window_step":
        rows = 0.87 * B * (W + S) if case["ragged"] else B * (W + S)  # a ring that is still filling has fewer
        return {"bytes": 2 * rows * Hkv * d * e + 2 * B * (H + 2 * Hkv) * d * e, "flops": 4 * rows * H * d}
    q, kv = H * tokens * d * e, Hkv * tokens * d * e
    pairs = H * mean(lambda x: _pairs(x, W, S))
    if op == "window_forward":
        return {"bytes": 2 * q + 2 * kv + 4 * H * tokens, "flops": 4 * d * pairs}
    return {"bytes": 4 * q + 4 * kv + 4 * H * tokens, "flops": 10 * d * pairs}


# --------------------------------------------------------------------------- definitions in 64 bits
def _gates64(case, g, rate):
    if case["gate"] == "given":
        return g, torch.ones_like(g)
    sg = 1 / (1 + torch.exp(-g))
    if case["gate"] == "sigmoid":
        return sg, 1 / (1 + torch.exp(g))
    u = rate.double() * sg
    return torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def _exact_gated_forward(s):
    case, n = s["case"], s["case"]["n"]
    h, L = s["state"].double(), s["lengths"]
    y = torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
    for t in range(n):
        a, f = _gates64(case, s["g"][:, t].double(), s["rate"])
        new = a * h + f * s["x"][:, t].double()
        if L is None:
            h = y[:, t] = new
        else:
            live = (t < L)[:, None]
            h = torch.where(live, new, h)
            y[:, t] = torch.where(live, new, 0.0)
    return y, h


def _exact_gated_backward(s):
    case, n, L = s["case"], s["case"]["n"], s["lengths"]
    c = s["dstate"].double()
    dx = torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
    dg = torch.zeros_like(dx)
    dr = torch.zeros(case["d"], device="cuda", dtype=torch.float64)
    for t in reversed(range(n)):
        x, g = s["x"][:, t].double(), s["g"][:, t].double()
        a, f = _gates64(case, g, s["rate"])
        before = s["y"][:, t - 1].double() if t else s["state"].double()
        gh = s["dy"][:, t].double() + c
        if case["gate"] == "rate":
            sg = 1 / (1 + torch.exp(-g))
            # b = f x, f = sqrt(1 - a^2), a = exp(-u): df/du = a^2 / f, da/du = -a
            du = gh * x * a * a / f - gh * before * a
            grad_g, grad_r = du * s["rate"].double() * sg * (1 - sg), du * sg
        else:
            grad_a = gh * before if case["gate"] == "given" else gh * (before - x)
            grad_g, grad_r = grad_a if case["gate"] == "given" else grad_a * a * f, None
        live = torch.ones_like(c, dtype=torch.bool) if L is None else (t < L)[:, None].expand_as(c)
        dx[:, t], dg[:, t] = torch.where(live, gh * f, 0.0), torch.where(live, grad_g, 0.0)
        if grad_r is not None:
            dr += torch.where(live, grad_r, 0.0).sum(0)
        c = torch.where(live, a * gh, c)
    return (dx, dg, c) + ((dr,) if case["gate"] == "rate" else ())


def _exact_gated_step(s):
    a, f = _gates64(s["case"], s["g"].double(), s["rate"])
    h = a * s["state"].double() + f * s["x"].double()
    if s["lengths"] is None:
        return h, h.clone()
    live = s["lengths"].bool()[:, None]
    return torch.where(live, h, s["y"].double()), torch.where(live, h, s["next"].double())


def _exact_window(s, backward):
    """Every sequence and key/value head by itself, 512 queries at a time against all keys they can reach."""
    case = s["case"]
    B, H, Hkv, n, d, W, S = (case[x] for x in ("B", "H", "Hkv", "n", "d", "window", "sinks"))
    G, scale = H // Hkv, 1 / math.sqrt(d)
    new = lambda *z: torch.zeros(*z, device="cuda", dtype=torch.float64)  # noqa: E731
    o, lse = new(B, H, n, d), new(B, H, n)
    dq, dk, dv = (new(B, H, n, d), new(B, Hkv, n, d), new(B, Hkv, n, d)) if backward else (None,) * 3
    for b in range(B):
        L = n if s["lengths"] is None else int(s["lengths"][b])
        for r0 in range(0, L, 512):
            r1 = min(L, r0 + 512)
            lo = max(0, r0 - W + 1)
            j = torch.cat([torch.arange(min(S, lo), device="cuda"), torch.arange(lo, r1, device="cuda")])
            p = torch.arange(r0, r1, device="cuda")[:, None]
            sees = (j <= p) & ((j > p - W) | (j < S))
            for hk in range(Hkv):
                hs = slice(hk * G, hk * G + G)
                q = s["q"][b, hs, r0:r1].double()
                k, v = s["k"][b, hk, j].double(), s["v"][b, hk, j].double()
                sc = torch.where(sees, q @ k.T * scale, -math.inf)
                if not backward:
                    z = torch.logsumexp(sc, -1)
                    lse[b, hs, r0:r1] = z
                    o[b, hs, r0:r1] = torch.exp(sc - z[..., None]) @ v
                    continue
                P = torch.exp(sc - s["lse"][b, hs, r0:r1].double()[..., None])
                g = s["do"][b, hs, r0:r1].double()
                D = torch.einsum("hnd,hnd->hn", g, s["o"][b, hs, r0:r1].double())
                dS = P * (g @ v.T - D[..., None]) * scale
                dq[b, hs, r0:r1] = dS @ k
                dk[b, hk, j] += torch.einsum("hnj,hnd->jd", dS, q)
                dv[b, hk, j] += torch.einsum("hnj,hnd->jd", P, g)
    return (dq, dk, dv) if backward else (o, lse)


def _exact_window_step(s):
    case = s["case"]
    B, H, Hkv, d, W, S = (case[x] for x in ("B", "H", "Hkv", "d", "window", "sinks"))
    o, kc, vc = s["o"].double(), s["kc"].double(), s["vc"].double()
    for b in range(B):
        p = int(s["pos"][b])
        if p < 0:
            continue
        at = p if p < S else S + (p - S) % W
        kc[b, :, at], vc[b, :, at] = s["k"][b].double(), s["v"][b].double()
        m = min(p + 1, S + W)
        for hk in range(Hkv):
            hs = slice(hk * (H // Hkv), (hk + 1) * (H // Hkv))
            P = torch.softmax(s["q"][b, hs].double() @ kc[b, hk, :m].T / math.sqrt(d), -1)
            o[b, hs] = P @ vc[b, hk, :m]
    return o, kc, vc


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated_forward":
        return _exact_gated_forward(s)
    if op == "gated_backward":
        return _exact_gated_backward(s)
    if op == "gated_step":
        return _exact_gated_step(s)
    if op in ("window_forward", "window_backward"):
        return _exact_window(s, op == "window_backward")
    return _exact_window_step(s)
