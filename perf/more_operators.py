"""Workloads of the operators of a selective state space layer: the short causal
convolution, the selective scan, and the norm over groups of channels with its
activation.  Inputs, the plain form of each operator, its definition in 64 bits, and the
bytes and operations it cannot do without.

Operators ("op" of a case):
  conv_forward, conv_backward, conv_step: y_t = act(sum_i w_i x_{t-(w-1)+i} + bias) per channel
  ssm_forward, ssm_backward, ssm_step:
      h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t^T,  y_t = C_t^T h_t + D x_t  per head
  norm_forward, norm_backward: each token's groups of channels normalised, scaled, shifted,
      through an activation or times an activated gate
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"


# --------------------------------------------------------------------------- cases
def _conv(op, B, n, d, width, act, dtype, ragged=False, name=None):
    c = {"op": op, "B": B, "n": n, "d": d, "width": width, "act": act, "dtype": dtype, "ragged": ragged}
    return {"name": name, **c} if name else c


def _ssm(op, B, n, H, G, P, N, softplus, dtype, ragged=False, name=None):
    c = {"op": op, "B": B, "n": n, "H": H, "G": G, "P": P, "N": N, "softplus": softplus, "dtype": dtype, "ragged": ragged}
    return {"name": name, **c} if name else c


def _norm(op, B, n, d, groups, center, gate, act, dtype, ragged=False, name=None):
    c = {"op": op, "B": B, "n": n, "d": d, "groups": groups, "center": center, "gate": gate, "act": act, "dtype": dtype,
         "ragged": ragged}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of a serving batch of 64 streams: 64 heads of 64 channels, B and C of 128
        _conv("conv_step", 64, 1, 4352, 4, "silu", BF16, name="conv_step_b64_d4352"),
        # padded batch of sequences of different lengths, an odd width, full precision
        _conv("conv_forward", 3, 5003, 1001, 3, "none", F32, ragged=True, name="conv_fwd_ragged_f32_n5003_d1001"),
        # one long sequence (prefill or long-context training)
        _conv("conv_forward", 1, 32768, 4352, 4, "silu", BF16, name="conv_fwd_n32768_d4352"),
        # training step of a wide layer, with the gradient of its filters
        _conv("conv_backward", 2, 8192, 4352, 4, "silu", BF16, name="conv_bwd_b2_n8192_d4352"),
        # one token of one stream: nothing but latency
        _ssm("ssm_step", 1, 1, 32, 1, 64, 128, True, BF16, name="ssm_step_b1_h32_p64_s128"),
        # a serving batch of 128 streams, some of them idle
        _ssm("ssm_step", 128, 1, 64, 1, 64, 128, True, BF16, ragged=True, name="ssm_step_b128_h64_p64_s128"),
        # training or prefill of a small layer, 8 heads of 64 channels
        _ssm("ssm_forward", 4, 2048, 8, 1, 64, 64, True, BF16, name="ssm_fwd_b4_n2048_h8_p64_s64"),
        # long prefill of a wide layer
        _ssm("ssm_forward", 1, 16384, 64, 1, 64, 128, True, BF16, name="ssm_fwd_n16384_h64_p64_s128"),
        # training on a padded batch in full precision, odd sizes, two groups of heads
        _ssm("ssm_backward", 3, 1501, 6, 2, 48, 40, False, F32, ragged=True, name="ssm_bwd_ragged_f32_n1501_h6_p48_s40"),
        # training step of a wide layer on long sequences
        _ssm("ssm_backward", 2, 8192, 32, 1, 64, 128, True, BF16, name="ssm_bwd_b2_n8192_h32_p64_s128"),
        # the norm behind the scan, times its activated gate, a prompt of a wide layer
        _norm("norm_forward", 1, 16384, 4096, 64, True, "after", "silu", BF16, name="norm_fwd_n16384_d4096_g64"),
        # training step: the gate goes in before the norm, one group, no mean
        _norm("norm_backward", 2, 8192, 4096, 1, False, "before", "silu", BF16, name="norm_bwd_b2_n8192_d4096_g1"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_forward", "conv_backward", "conv_step", "ssm_forward", "ssm_forward", "ssm_backward",
                     "ssm_backward", "ssm_step", "norm_forward", "norm_backward"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    ragged = rng.random() < 0.4
    if op.startswith("conv"):
        width, act = rng.choice([2, 3, 4, 4, 4]), rng.choice(["none", "silu", "silu"])
        if op == "conv_step":
            return _conv(op, _log_int(rng, 1, 256), 1, _log_int(rng, 64, 8192), width, act, dtype, ragged)
        while True:
            B, n, d = _log_int(rng, 1, 16), _log_int(rng, 1, 32768), _log_int(rng, 33, 8192)
            if rng.random() < 0.5:
                d = (d + 63) // 64 * 64
            if B * n * d * (2 if dtype == F32 else 1) <= 1 << 26:
                return _conv(op, B, n, d, width, act, dtype, ragged)
    if op.startswith("norm"):
        gate, act = rng.choice([("none", "none"), ("none", "silu"), ("after", "silu"), ("before", "silu")])
        while True:
            groups, B, n = rng.choice([1, 1, 2, 8, 32, 64]), _log_int(rng, 1, 16), _log_int(rng, 1, 32768)
            d = groups * _log_int(rng, 8, 8192 // groups)
            if B * n * d * (2 if dtype == F32 else 1) <= 1 << 26:
                return _norm(op, B, n, d, groups, rng.random() < 0.5, gate, act, dtype, ragged)
    G = rng.choice([1, 1, 1, 2, 8])
    H = G * rng.choice([1, 2, 3, 4, 8])
    P, N = rng.choice([32, 48, 64, 64, 64, 128]), rng.choice([16, 40, 64, 64, 128, 128])
    softplus = rng.random() < 0.7
    if op == "ssm_step":
        return _ssm(op, _log_int(rng, 1, 128), 1, H, G, P, N, softplus, dtype, ragged)
    while True:
        B, n = _log_int(rng, 1, 8), _log_int(rng, 1, 16384)
        products = (4 if op == "ssm_forward" else 10) * B * H * n * N * P
        # full precision does its products at the rate of fp32 arithmetic
        if products <= (4e10 if dtype == BF16 else 4e9) and B * H * n <= 1 << 20:
            return _ssm(op, B, n, H, G, P, N, softplus, dtype, ragged)


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


def _live(case, gen):
    """A ragged serving batch has idle slots."""
    return (torch.rand(case["B"], generator=gen, device="cuda") < 0.8).to(torch.int32) if case["ragged"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    dt = _dt(case)
    op, B, n = case["op"], case["B"], case["n"]
    step, back = op.endswith("step"), op.endswith("backward")

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": dict(case)}
    if op.startswith("conv"):
        d, w = case["d"], case["width"]
        s["x"] = randn(*((B, d) if step else (B, n, d))).to(dt)
        s["weight"], s["bias"] = randn(d, w) / math.sqrt(w), 0.1 * randn(d)
        s["state"] = randn(B, w - 1, d).to(dt)
        if step:
            s["lengths"] = _live(case, gen)
            s["y"] = torch.zeros_like(s["x"])
            return s
        s["lengths"] = _lengths(case, gen, n)
        if back:
            s["dy"], s["dstate"] = randn(B, n, d).to(dt), randn(B, w - 1, d).to(dt)
        return s
    if op.startswith("norm"):
        d = case["d"]
        s["x"] = (randn(B, n, d) * torch.exp(randn(B, n, 1)) + 0.3).to(dt)
        s["gate"] = randn(B, n, d).to(dt) if case["gate"] != "none" else None
        s["weight"], s["bias"] = 1 + 0.2 * randn(d), 0.2 * randn(d)
        s["lengths"] = _lengths(case, gen, n)
        if back:
            s["dy"] = randn(B, n, d).to(dt)
        return s
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    # x, B and C are slices of the convolution's output, tokens outside heads
    wide = randn(B, n, H * P + 2 * G * N).to(dt)
    s["wide"] = wide
    s["x"] = wide[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
    s["Bt"] = wide[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
    s["Ct"] = wide[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2)
    # steps of 0.001 to 0.1 and rates of 1 to 16, as layers of this kind start from
    u = lambda *z: torch.rand(*z, generator=gen, device="cuda")  # noqa: E731
    at = torch.exp(u(H) * math.log(100.0) + math.log(0.001))
    s["A"] = -(1 + 15 * u(H))
    s["D"] = 1 + 0.1 * randn(H)
    if case["softplus"]:
        s["bias"] = at + torch.log(-torch.expm1(-at))
        s["dt"] = (0.5 * randn(B, n, H)).to(dt).transpose(1, 2)
    else:
        s["bias"] = None
        s["dt"] = (at * torch.exp(0.5 * randn(B, n, H))).to(dt).transpose(1, 2)
    s["state"] = randn(B, H, N, P)
    if step:
        for k in ("x", "Bt", "Ct", "dt"):
            s[k] = s[k][:, :, 0]
        s["lengths"] = _live(case, gen)
        s["y"] = torch.zeros(B, H, P, device="cuda", dtype=dt)
        return s
    s["lengths"] = _lengths(case, gen, n)
    if back:
        s["dy"] = randn(B, n, H, P).to(dt).transpose(1, 2)
        s["dstate"] = randn(B, H, N, P)
    return s


# --------------------------------------------------------------------------- plain forms
def _valid(s, n):
    """[B, n]: token t is below its sequence's length."""
    if s["lengths"] is None:
        return None
    return torch.arange(n, device="cuda") < s["lengths"][:, None]


def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _held(s):
    """Where the last w - 1 inputs of each sequence lie behind the state that came before it."""
    case = s["case"]
    L = s["lengths"].long() if s["lengths"] is not None else torch.full((case["B"],), case["n"], device="cuda")
    return (L[:, None] + torch.arange(case["width"] - 1, device="cuda"))[..., None].expand(-1, -1, case["d"])


def _conv_pre(s):
    xs = torch.cat([s["state"], s["x"]], 1).float()
    taps = xs.unfold(1, s["case"]["width"], 1)  # [B, n, d, w]
    return xs, taps, (taps * s["weight"]).sum(-1) + s["bias"]


def _conv_forward(s):
    xs, _, y = _conv_pre(s)
    if s["case"]["act"] == "silu":
        y = _silu(y)
    ok = _valid(s, s["case"]["n"])
    if ok is not None:
        y = torch.where(ok[..., None], y, 0.0)
    return y.to(s["x"].dtype), xs.gather(1, _held(s)).to(s["x"].dtype)


def _conv_backward(s):
    case, dt = s["case"], s["x"].dtype
    n, w = case["n"], case["width"]
    xs, taps, pre = _conv_pre(s)
    g = s["dy"].float()
    if case["act"] == "silu":
        g = g * _dsilu(pre)
    ok = _valid(s, n)
    if ok is not None:
        g = torch.where(ok[..., None], g, 0.0)
    dw = (g[..., None] * taps).sum((0, 1))
    ahead = torch.nn.functional.pad(g, (0, 0, w - 1, w - 1)).unfold(1, w, 1)  # g_{i-(w-1)} .. g_i for input i
    dxs = (ahead * s["weight"].flip(1)).sum(-1)
    dxs = dxs.scatter_add(1, _held(s), s["dstate"].float())
    dx = dxs[:, w - 1:]
    if ok is not None:
        dx = torch.where(ok[..., None], dx, 0.0)
    return dx.to(dt), dw, g.sum((0, 1)), dxs[:, :w - 1].to(dt)


def _conv_step(s):
    xs = torch.cat([s["state"], s["x"][:, None]], 1)
    y = (xs.float() * s["weight"].t()).sum(1) + s["bias"]
    if s["case"]["act"] == "silu":
        y = _silu(y)
    y, state = y.to(s["x"].dtype), xs[:, 1:]
    if s["lengths"] is not None:
        live = s["lengths"][:, None] > 0
        y, state = torch.where(live, y, s["y"]), torch.where(live[..., None], state, s["state"])
    s["state"].copy_(state)
    return y, s["state"]


def _steps(s, ok=None):
    """dt_t in 32 bits (zero behind the sequence) and what it has of a slope in the raw one."""
    raw = s["dt"].float()
    if s["case"]["softplus"]:
        raw = raw + s["bias"].view(-1, *(1,) * (raw.dim() - 2))
        dt, slope = torch.nn.functional.softplus(raw, threshold=80.0), torch.sigmoid(raw)
    else:
        dt, slope = raw, torch.ones_like(raw)
    if ok is not None:
        dt, slope = torch.where(ok[:, None], dt, 0.0), torch.where(ok[:, None], slope, 0.0)
    return dt, slope


CHUNK = 128


def _chunks(x, G, c, nc, ok):
    """[B, heads, n, w] to [B, G, heads / G, chunks, c, w] in 32 bits, zero behind the sequence."""
    x = x.float()
    if ok is not None:
        x = torch.where(ok[:, None, :, None], x, 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, nc * c - x.shape[2]))
    return x.reshape(x.shape[0], G, x.shape[1] // G, nc, c, x.shape[-1])


class _Chunked:
    """What both directions of the scan share: the chunks, and the decays inside and between them."""

    def __init__(self, s):
        case = s["case"]
        self.B, self.n, self.H, self.G, self.P, self.N = (case[k] for k in ("B", "n", "H", "G", "P", "N"))
        self.c = c = min(CHUNK, self.n)
        self.nc = nc = -(-self.n // c)
        self.ok = _valid(s, self.n)
        dt, self.slope = _steps(s, self.ok)
        self.dt = _chunks(dt[..., None], self.G, c, nc, None)[..., 0]  # [B, G, R, nc, c]
        self.A = s["A"].view(self.G, -1, 1, 1)
        self.x = _chunks(s["x"], self.G, c, nc, self.ok)
        self.b = _chunks(s["Bt"], self.G, c, nc, self.ok)
        self.cc = _chunks(s["Ct"], self.G, c, nc, self.ok)
        # positions along the decay: 64 bits, their differences are what counts
        self.pos = torch.cumsum(self.dt.double() * self.A.double(), -1)
        self.end = self.pos[..., -1]
        keep = torch.ones(c, c, device="cuda", dtype=torch.bool).tril()
        self.L = torch.where(keep, torch.exp((self.pos[..., :, None] - self.pos[..., None, :]).float()), 0.0)
        self.to = torch.exp(self.pos.float())[..., None]  # from the chunk's start to the token
        self.rest = torch.exp((self.end[..., None] - self.pos).float())[..., None]  # from the token to its end
        far = torch.cumsum(self.end, -1)
        hop = far[..., :, None] - self.end[..., :, None] - far[..., None, :]  # what chunk j's end lost at i's start
        before = torch.ones(nc, nc, device="cuda", dtype=torch.bool).tril(-1)
        self.hop = torch.where(before, torch.exp(hop.float()), 0.0)
        self.start = torch.exp((far - self.end).float())[..., None, None]
        self.finish = torch.exp((far[..., -1:] - far).float())[..., None, None]
        self.all = torch.exp(far[..., -1].float())[..., None, None]
        self.state = s["state"].reshape(self.B, self.G, -1, self.N, self.P)
        add = (self.b * (self.dt * self.rest[..., 0])[..., None]).transpose(-1, -2) @ self.x  # [B, G, R, nc, N, P]
        self.before = (self.hop @ add.flatten(-2)).unflatten(-1, (self.N, self.P)) + self.start * self.state[:, :, :, None]
        self.last = (self.finish * add).sum(3) + self.all * self.state

    def whole(self, x):
        """[B, G, heads / G, chunks, c, w] to [B, heads, n, w]."""
        return x.reshape(self.B, -1, self.nc * self.c, x.shape[-1])[:, :, :self.n]


def _ssm_forward(s):
    k = _Chunked(s)
    y = ((k.cc @ k.b.transpose(-1, -2)) * k.L * k.dt[..., None, :]) @ k.x + k.to * (k.cc @ k.before)
    y = k.whole(y + s["D"].view(k.G, -1, 1, 1, 1) * k.x)
    return y.to(s["x"].dtype), k.last.reshape(s["state"].shape).contiguous()


def _after(x):
    """Sums of what follows, the element itself among them, along the last dimension: 64 bits."""
    return x.flip(-1).cumsum(-1, dtype=torch.float64).flip(-1)


def _ssm_backward(s):
    case, dt = s["case"], s["x"].dtype
    k = _Chunked(s)
    dy = _chunks(s["dy"], k.G, k.c, k.nc, k.ok)
    ds = s["dstate"].reshape(k.state.shape)
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    # the states' gradients at the chunks' ends
    add = T(k.cc * k.to) @ dy
    back = (T(k.hop) @ add.flatten(-2)).unflatten(-1, (k.N, k.P)) + k.finish * ds[:, :, :, None]
    first = (k.start * add).sum(3) + k.all * ds
    M = (k.cc @ T(k.b)) * k.L
    S = (dy @ T(k.x)) * k.L
    E = M * (dy @ T(k.x))
    gb = k.rest * (k.b @ back)  # [.., c, P]
    hy = k.to * (k.cc @ k.before)
    dxt = T(M) @ dy + gb
    D = s["D"].view(k.G, -1, 1, 1, 1)
    dx = k.dt[..., None] * dxt + D * dy
    dB = k.dt[..., None] * (T(S) @ k.cc + k.rest * (k.x @ T(back)))
    dC = (S * k.dt[..., None, :]) @ k.b + k.to * (dy @ T(k.before))
    dB, dC = dB.sum(2, keepdim=True), dC.sum(2, keepdim=True)
    # the gradient of log decays: what passes the token from those before it to those behind
    inside = _after((E * k.dt[..., None, :]).sum(-1)) - _after(E.sum(-2) * k.dt)
    u = (k.x * gb).sum(-1)
    w = (dy * hy).sum(-1)
    from_before = (u * k.dt).cumsum(-1, dtype=torch.float64) - u * k.dt
    through = (torch.exp(k.end.float()) * (back * k.before).sum((-1, -2)))[..., None]
    da = (inside + _after(w) + from_before + through).float()
    d_dt = k.A * da + E.sum(-2) + u
    d_dt = k.whole(d_dt[..., None])[..., 0] * k.slope
    dA = (da * k.dt).sum((0, 3, 4), dtype=torch.float64).float().view(-1)
    dD = (dy * k.x).sum((0, 3, 4, 5)).view(-1)
    out = [k.whole(dx).to(dt), d_dt.to(dt), dA, k.whole(dB).to(dt), k.whole(dC).to(dt), dD]
    if case["softplus"]:
        out.append(d_dt.sum((0, 2)))
    return (*out, first.reshape(s["state"].shape).contiguous())


def _ssm_step(s):
    case = s["case"]
    R = case["H"] // case["G"]
    dt, _ = _steps(s)
    b, c = (s[k].float().repeat_interleave(R, 1) for k in ("Bt", "Ct"))
    x = s["x"].float()
    h = torch.exp(dt * s["A"])[..., None, None] * s["state"] + b[..., None] * (dt[..., None] * x)[:, :, None]
    y = ((c[..., None] * h).sum(2) + s["D"][:, None] * x).to(s["x"].dtype)
    if s["lengths"] is not None:
        live = s["lengths"][:, None, None] > 0
        y, h = torch.where(live, y, s["y"]), torch.where(live[..., None], h, s["state"])
    s["state"].copy_(h)
    return y, s["state"]


def _normalised(s):
    """The norm's input, itself normalised, and 1 / its deviation, by groups [B, n, groups, d / groups]."""
    case = s["case"]
    u = s["x"].float()
    if case["gate"] == "before":
        u = u * _silu(s["gate"].float())
    u = u.unflatten(-1, (case["groups"], -1))
    if case["center"]:
        u = u - u.mean(-1, keepdim=True)
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    return u * r, r


def _norm_forward(s):
    case = s["case"]
    v = _normalised(s)[0].flatten(-2) * s["weight"] + s["bias"]
    if case["gate"] == "after":
        v = v * _silu(s["gate"].float())
    elif case["gate"] == "none" and case["act"] == "silu":
        v = _silu(v)
    ok = _valid(s, case["n"])
    return (v if ok is None else torch.where(ok[..., None], v, 0.0)).to(s["x"].dtype)


def _norm_backward(s):
    case, dt = s["case"], s["x"].dtype
    ok = _valid(s, case["n"])
    dy = s["dy"].float()
    if ok is not None:
        dy = torch.where(ok[..., None], dy, 0.0)
    z, r = _normalised(s)
    zf = z.flatten(-2)
    v = zf * s["weight"] + s["bias"]
    dgate = None
    if case["gate"] == "after":
        gate = s["gate"].float()
        dgate = dy * v * _dsilu(gate)
        dy = dy * _silu(gate)
    elif case["gate"] == "none" and case["act"] == "silu":
        dy = dy * _dsilu(v)
    dw, db = (dy * zf).sum((0, 1)), dy.sum((0, 1))
    g = (dy * s["weight"]).unflatten(-1, (case["groups"], -1))
    du = g - z * (g * z).mean(-1, keepdim=True)
    if case["center"]:
        du = du - g.mean(-1, keepdim=True)
    du = (du * r).flatten(-2)
    if case["gate"] == "before":
        gate = s["gate"].float()
        dgate = du * s["x"].float() * _dsilu(gate)
        du = du * _silu(gate)
    return (du.to(dt), dw, db) + (() if dgate is None else (dgate.to(dt),))


# --------------------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"conv_forward": _conv_forward, "conv_backward": _conv_backward, "conv_step": _conv_step,
                "ssm_forward": _ssm_forward, "ssm_backward": _ssm_backward, "ssm_step": _ssm_step,
                "norm_forward": _norm_forward, "norm_backward": _norm_backward}[op](s)
    import causal_prefix_scan_gb300 as hla
    if op == "conv_forward":
        return hla.conv_forward(s["x"], s["weight"], s["bias"], activation=case["act"], state_in=s["state"],
                                return_state=True, lengths=s["lengths"])
    if op == "conv_backward":
        if "ws" not in s:  # kept by the program from its first call on
            s["ws"] = hla.conv_workspace(s["x"], s["weight"])
        r = hla.conv_backward(s["x"], s["dy"], s["weight"], s["bias"], activation=case["act"], state_in=s["state"],
                              d_state_out=s["dstate"], want_dstate=True, lengths=s["lengths"], workspace=s["ws"])
        return r.dx, r.d_weight, r.d_bias, r.d_state_in
    if op == "conv_step":
        return hla.conv_step(s["state"], s["x"], s["weight"], s["bias"], activation=case["act"], lengths=s["lengths"],
                             out=s["y"]), s["state"]
    if op.startswith("norm"):
        kw = {"groups": case["groups"], "eps": 1e-5, "center": case["center"], "gate": s["gate"],
              "gate_first": case["gate"] == "before", "activation": case["act"], "lengths": s["lengths"]}
        if op == "norm_forward":
            return hla.norm_forward(s["x"], s["weight"], s["bias"], **kw)
        if "ws" not in s:
            s["ws"] = hla.norm_workspace(s["x"])
        r = hla.norm_backward(s["x"], s["dy"], s["weight"], s["bias"], workspace=s["ws"], **kw)
        return (r.dx, r.d_weight, r.d_bias) + (() if r.d_gate is None else (r.d_gate,))
    kw = {"D": s["D"], "dt_bias": s["bias"], "dt_softplus": case["softplus"], "lengths": s["lengths"]}
    if op == "ssm_step":
        return hla.ssm_step(s["state"], s["x"], s["dt"], s["A"], s["Bt"], s["Ct"], out=s["y"], **kw), s["state"]
    if "ws" not in s:
        s["ws"] = hla.ssm_workspace(s["x"], s["Bt"], backward=op == "ssm_backward")
    if op == "ssm_forward":
        return hla.ssm_forward(s["x"], s["dt"], s["A"], s["Bt"], s["Ct"], state_in=s["state"], return_state=True,
                               workspace=s["ws"], **kw)
    r = hla.ssm_backward(s["x"], s["dt"], s["A"], s["Bt"], s["Ct"], s["dy"], state_in=s["state"],
                         d_state_out=s["dstate"], want_dstate=True, workspace=s["ws"], **kw)
    return (r.dx, r.d_dt, r.dA, r.dB, r.dC, r.dD) + (() if r.d_dt_bias is None else (r.d_dt_bias,)) + (r.d_state_in,)


# --------------------------------------------------------------------------- floors
def work(case):
    e = 4 if case["dtype"] == F32 else 2
    B, n, op = case["B"], case["n"], case["op"]
    if op.endswith("step"):
        tokens = 0.8 * B if case["ragged"] else B  # idle slots
    elif case["ragged"]:  # the first sequence is whole, the others 5 % to all of it
        tokens = n + (B - 1) * n * 0.525
    else:
        tokens = B * n
    if op.startswith("conv"):
        d, w = case["d"], case["width"]
        N, held, par = tokens * d, B * (w - 1) * d * e, 4 * d * (w + 1)
        if op == "conv_step":
            return {"bytes": 2 * N * e + 2 * (w - 1) * N * e + par, "flops": 2 * w * N}
        if op == "conv_forward":
            return {"bytes": 2 * N * e + 2 * held + par, "flops": 2 * w * N}
        return {"bytes": 3 * N * e + 3 * held + 2 * par, "flops": 6 * w * N}
    if op.startswith("norm"):
        N = tokens * case["d"]
        gated = case["gate"] != "none"
        if op == "norm_forward":
            return {"bytes": (2 + gated) * N * e + 8 * case["d"], "flops": 8 * N}
        return {"bytes": (3 + 2 * gated) * N * e + 16 * case["d"], "flops": 16 * N}
    H, G, P, S = case["H"], case["G"], case["P"], case["N"]
    x, bc, dt, held = tokens * H * P * e, tokens * G * S * e, tokens * H * e, 4 * B * H * S * P
    if op == "ssm_step":
        return {"bytes": 2 * x + 2 * bc + dt + 8 * tokens * H * S * P, "flops": 4 * tokens * H * S * P}
    if op == "ssm_forward":
        return {"bytes": 2 * x + 2 * bc + dt + 2 * held, "flops": 4 * tokens * H * S * P}
    return {"bytes": 3 * x + 4 * bc + 2 * dt + 3 * held, "flops": 10 * tokens * H * S * P}


# --------------------------------------------------------------------------- definitions in 64 bits
def _new(*shape):
    return torch.zeros(*shape, device="cuda", dtype=torch.float64)


def _len(s, b):
    return s["case"]["n"] if s["lengths"] is None else int(s["lengths"][b])


def _sig64(x):
    return 1 / (1 + torch.exp(-x))


def _exact_conv(s, backward):
    """Every sequence by itself, one tap after the other."""
    case = s["case"]
    B, n, d, w = (case[k] for k in ("B", "n", "d", "width"))
    y, dx, dw, db = _new(B, n, d), _new(B, n, d), _new(d, w), _new(d)
    held, dheld = _new(B, w - 1, d), _new(B, w - 1, d)
    for b in range(B):
        L = _len(s, b)
        xs = torch.cat([s["state"][b], s["x"][b, :L]]).double()
        pre = s["bias"].double() + sum(s["weight"][:, i].double() * xs[i:i + L] for i in range(w))
        held[b] = xs[L:]
        g = _sig64(pre)
        silu = case["act"] == "silu"
        y[b, :L] = pre * g if silu else pre
        if not backward:
            continue
        dp = s["dy"][b, :L].double()
        if silu:
            dp = dp * (g + pre * g * (1 - g))
        dxs = torch.zeros_like(xs)
        for i in range(w):
            dxs[i:i + L] += dp * s["weight"][:, i].double()
            dw[:, i] += (dp * xs[i:i + L]).sum(0)
        dxs[L:] += s["dstate"][b].double()
        db += dp.sum(0)
        dheld[b], dx[b, :L] = dxs[:w - 1], dxs[w - 1:]
    return (dx, dw, db, dheld) if backward else (y, held)


def _exact_conv_step(s):
    state, y = s["state"].double(), s["y"].double()
    xs = torch.cat([state, s["x"].double()[:, None]], 1)
    pre = torch.einsum("bid,di->bd", xs, s["weight"].double()) + s["bias"].double()
    out = pre * _sig64(pre) if s["case"]["act"] == "silu" else pre
    for b in range(s["case"]["B"]):
        if s["lengths"] is None or int(s["lengths"][b]):
            y[b], state[b] = out[b], xs[b, 1:]
    return y, state


def _steps64(s, t=None):
    raw = s["dt"].double() if t is None else s["dt"][:, :, t].double()
    if not s["case"]["softplus"]:
        return raw, torch.ones_like(raw)
    raw = raw + s["bias"].double()
    return torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), _sig64(raw)


class _Tokens:
    """The recurrence one token at a time, all sequences at once."""

    def __init__(self, s):
        self.s, self.R = s, s["case"]["H"] // s["case"]["G"]
        self.A, self.D = s["A"].double(), s["D"].double()

    def at(self, t):
        s = self.s
        dt, slope = _steps64(s, t)
        wide = lambda k: s[k][:, :, t].double().repeat_interleave(self.R, 1)  # noqa: E731
        live = torch.ones_like(dt) if s["lengths"] is None else (t < s["lengths"]).double()[:, None].expand_as(dt)
        zero = lambda x: torch.where(live[..., None] > 0, x, 0.0)  # noqa: E731
        dt, slope = dt * live, slope * live
        return dt, slope, torch.exp(dt * self.A)[..., None, None], zero(s["x"][:, :, t].double()), zero(wide("Bt")), \
            zero(wide("Ct")), live

    def on(self, h, dt, decay, x, b):
        return decay * h + (dt[..., None] * b)[..., None] * x[:, :, None]


def _exact_ssm_forward(s):
    k, n = _Tokens(s), s["case"]["n"]
    h, y = s["state"].double(), _new(*s["x"].shape)
    for t in range(n):
        dt, _, decay, x, b, c, _ = k.at(t)
        h = k.on(h, dt, decay, x, b)
        y[:, :, t] = (c[..., None] * h).sum(2) + k.D[:, None] * x
    return y, h


def _exact_ssm_backward(s):
    case, k = s["case"], _Tokens(s)
    B, n, H, G, P, N = (case[x] for x in ("B", "n", "H", "G", "P", "N"))
    dx, ddt, dB, dC = _new(B, H, n, P), _new(B, H, n), _new(B, G, n, N), _new(B, G, n, N)
    dA, dD, dbias = _new(H), _new(H), _new(H)
    step = 64
    kept, h = [], s["state"].double()
    for t in range(n):  # the states at every 64th token
        if t % step == 0:
            kept.append(h)
        dt, _, decay, x, b, _, _ = k.at(t)
        h = k.on(h, dt, decay, x, b)
    g = s["dstate"].double()
    for t0 in reversed(range(0, n, step)):
        hs, at = [kept[t0 // step]], []
        for t in range(t0, min(n, t0 + step)):
            at.append(k.at(t))
            dt, _, decay, x, b, _, _ = at[-1]
            hs.append(k.on(hs[-1], dt, decay, x, b))
        for t in reversed(range(t0, min(n, t0 + step))):
            dt, slope, decay, x, b, c, live = at[t - t0]
            before, h = hs[t - t0], hs[t - t0 + 1]
            dy = torch.where(live[..., None] > 0, s["dy"][:, :, t].double(), 0.0)
            g = g + c[..., None] * dy[:, :, None]
            dC[:, :, t] = (h * dy[:, :, None]).sum(-1).view(B, G, -1, N).sum(2)
            gb = (g * b[..., None]).sum(2)
            dx[:, :, t] = dt[..., None] * gb + k.D[:, None] * dy
            dB[:, :, t] = (dt[..., None] * (g * x[:, :, None]).sum(-1)).view(B, G, -1, N).sum(2)
            da = (g * decay * before).sum((-1, -2))
            d = (k.A * da + (gb * x).sum(-1)) * slope
            ddt[:, :, t] = d
            dA += (da * dt).sum(0)
            dD += (dy * x).sum((0, -1))
            dbias += d.sum(0)
            g = decay * g
    return (dx, ddt, dA, dB, dC, dD) + ((dbias,) if case["softplus"] else ()) + (g,)


def _exact_ssm_step(s):
    case = s["case"]
    R = case["H"] // case["G"]
    dt, _ = _steps64(s)
    h, y = s["state"].double(), s["y"].double()
    for b in range(case["B"]):
        if s["lengths"] is not None and not int(s["lengths"][b]):
            continue
        x, bt, ct = s["x"][b].double(), s["Bt"][b].double().repeat_interleave(R, 0), s["Ct"][b].double().repeat_interleave(R, 0)
        h[b] = torch.exp(dt[b] * s["A"].double())[:, None, None] * h[b] + torch.einsum("h,hn,hp->hnp", dt[b], bt, x)
        y[b] = torch.einsum("hn,hnp->hp", ct, h[b]) + s["D"].double()[:, None] * x
    return y, h


def _exact_norm(s, backward):
    """Every sequence by itself; the gradient by the quotient rule on sums of squares."""
    case = s["case"]
    B, n, d, m = case["B"], case["n"], case["d"], case["d"] // case["groups"]
    w, bias = s["weight"].double(), s["bias"].double()
    y, dx, dg, dw, db = _new(B, n, d), _new(B, n, d), _new(B, n, d), _new(d), _new(d)
    for b in range(B):
        L = _len(s, b)
        x = s["x"][b, :L].double()
        gate = s["gate"][b, :L].double() if s["gate"] is not None else None
        sg = _sig64(gate) if gate is not None else None
        act, slope = (gate * sg, sg + gate * sg * (1 - sg)) if gate is not None else (None, None)
        u = x * act if case["gate"] == "before" else x
        ug = u.view(L, -1, m)
        mean = ug.mean(-1, keepdim=True) if case["center"] else 0.0
        q = ((ug - mean) ** 2).mean(-1, keepdim=True) + 1e-5
        z = ((ug - mean) / q.sqrt()).view(L, d)
        v = z * w + bias
        sv = _sig64(v)
        f = v * act if case["gate"] == "after" else v * sv if case["gate"] == "none" and case["act"] == "silu" else v
        y[b, :L] = f
        if not backward:
            continue
        dv = s["dy"][b, :L].double()
        if case["gate"] == "after":
            dg[b, :L] = dv * v * slope
            dv = dv * act
        elif case["gate"] == "none" and case["act"] == "silu":
            dv = dv * (sv + v * sv * (1 - sv))
        dw += (dv * z).sum(0)
        db += dv.sum(0)
        dz = (dv * w).view(L, -1, m)
        c = ug - mean
        dc = dz / q.sqrt() - c * (dz * c).mean(-1, keepdim=True) / (q * q.sqrt())
        if case["center"]:
            dc = dc - dc.mean(-1, keepdim=True)
        du = dc.reshape(L, d)
        if case["gate"] == "before":
            dg[b, :L] = du * x * slope
            du = du * act
        dx[b, :L] = du
    if not backward:
        return y
    return (dx, dw, db) + ((dg,) if s["gate"] is not None else ())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv_forward", "conv_backward"):
        return _exact_conv(s, op == "conv_backward")
    if op == "conv_step":
        return _exact_conv_step(s)
    if op == "ssm_forward":
        return _exact_ssm_forward(s)
    if op == "ssm_backward":
        return _exact_ssm_backward(s)
    if op == "ssm_step":
        return _exact_ssm_step(s)
    return _exact_norm(s, op == "norm_backward")
