"""Plain 64-bit forms of the selective state space layer's operators, with bounds on what
rounding may do to a kernel's results.

Bounds.  u = 2^-24 is half a step of fp32; a bound is a number of u times the same form on
absolute values (every product positive), and the store adds half a step of the element type.
  Sigmoid: the exponential's argument is off by 2 |z| u, its result by 4 u, the quotient by 4 u:
      (16 + 2 |z|) u with the sum in between.
  Convolution: width + 1 roundings of the sum of absolute products, then the activation (its slope
      is below 1.1).
  Scan: 2^(s_t - s_j) is off by 8 u inside a chunk whatever the distance, by 16 u more for each
      chunk between; a step by 32 u, which moves a decay e^-z by 32 z u (z e^-z < 0.4 of the
      undecayed term; 512 covers z up to 16, and what lies behind is below 2^-23 of it);
      sums of k terms by k u.  On the tensor cores bf16 operands are exact; the weights M, S are
      rounded to bf16 once (half a step 2^-9 of the value below a power of two, 2^-8 at most) and so
      is a state that enters y, dx, dB, dC; a state that is kept, and what the gradients of dt, A and
      dt_bias take of it, enters in three bf16 parts, whose sum is the fp32 value.
      Underflow: a factor, or a part of a weighted operand, below 2^-126 is 0.  Each output is a sum of
      at most n N P (n + 1) products of such a factor with one element each of x, B, C, dy, a state,
      D, A and dt, so it moves by at most 2^-126 times that count and the largest elements: below
      1e-20 for every test here, and nothing but values of 1e-15 and less can tell.
  Gradient of the log decays: differences of sums over a chunk (of at most 128 tokens), so its
      bound takes those sums.
  Norm: sums of m terms, each statistic relative to the spread of u: mean(|u|) m u enters z
      through 1 / deviation.
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, bound, name):
    """|got - want| <= bound + the store's rounding."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, name
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    off = (got - want).abs()
    bad = off > bound
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound.clamp(min=1e-300)).max()):.3g} times the bound"


def sig(z):
    return torch.sigmoid(z)


def act(z, kind):
    return z * sig(z) if kind == "silu" else z


def slope(z, kind):
    g = sig(z)
    return g * (1 + z * (1 - g)) if kind == "silu" else torch.ones_like(z)


def e_sig(z):
    return (16 + 2 * z.abs()) * U


def live_rows(lengths, B, n, device):
    if lengths is None:
        return torch.ones(B, n, dtype=torch.bool, device=device)
    return torch.arange(n, device=device)[None] < lengths.clamp(0, n)[:, None]


# ------------------------------------------------------------------ convolution
def conv(x, weight, bias, kind, state=None, lengths=None, dy=None, dstate=None):
    """Dict of name -> (value, bound before the store's rounding)."""
    B, n, d = x.shape
    w = weight.shape[1]
    W = weight.double()
    b = torch.zeros(d, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    ok = live_rows(lengths, B, n, x.device)[..., None]
    L = ok[..., 0].sum(1)
    st = torch.zeros(B, w - 1, d, dtype=torch.float64, device=x.device) if state is None else state.double()
    xs = torch.cat([st, torch.where(ok, x.double(), 0.0)], 1)
    taps = torch.stack([xs[:, i:i + n] for i in range(w)], -1)
    pre, size = (taps * W).sum(-1) + b, (taps.abs() * W.abs()).sum(-1) + b.abs()
    e_pre = (w + 2) * U * size
    y = act(pre, kind)
    e_y = 1.1 * e_pre + (pre.abs() * e_sig(pre) + 2 * U * y.abs() if kind == "silu" else 0.0)
    at = (L[:, None] + torch.arange(w - 1, device=x.device))[..., None].expand(-1, -1, d)
    r = {"y": (torch.where(ok, y, 0.0), torch.where(ok, e_y, 0.0)), "state": (xs.gather(1, at), torch.zeros_like(st))}
    if dy is None:
        return r
    g = torch.where(ok, dy.double() * slope(pre, kind), 0.0)
    # the slope's own slope is below 0.6
    e_g = torch.where(ok, dy.double().abs() * ((0.6 * e_pre + (1 + pre.abs()) * (e_sig(pre) + 4 * U)) if kind == "silu" else 0.0), 0.0)

    def spread(t, weights):
        out = torch.zeros(B, n + w - 1, d, dtype=torch.float64, device=x.device)
        for i in range(w):
            out[:, i:i + n] += t * weights[:, i]
        return out

    dxs = spread(g, W)
    e = spread(e_g, W.abs()) + (w + 2) * U * spread(g.abs(), W.abs())
    if dstate is not None:
        dxs.scatter_add_(1, at, dstate.double())
        e.scatter_add_(1, at, 2 * U * dstate.double().abs())
    k = (B * n / 8 + 64) * U  # a run of 32 tokens, eight runs, then the tiles in eight rows: below n / 8 + 64 roundings
    ax = taps.abs()
    r["dx"] = (torch.where(ok, dxs[:, w - 1:], 0.0), torch.where(ok, e[:, w - 1:], 0.0))
    r["d_state_in"] = (dxs[:, :w - 1], e[:, :w - 1])
    r["d_weight"] = ((g[..., None] * taps).sum((0, 1)), ((e_g[..., None] + k * g.abs()[..., None]) * ax).sum((0, 1)))
    r["d_bias"] = (g.sum((0, 1)), (e_g + k * g.abs()).sum((0, 1)))
    return r


# ------------------------------------------------------------------ scan
def _steps(dt, dt_bias, softplus):
    raw = dt.double()
    if not softplus:
        return raw, torch.ones_like(raw)
    if dt_bias is not None:
        raw = raw + dt_bias.double()[None, :, None]
    return raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs())), sig(raw)


def _scan(x, dt, slope_, A, B, C, D, state, lengths, dy, dstate, size):
    """Values, or with `size` the same on absolute values: every term positive."""
    f = (lambda t: None if t is None else t.double().abs()) if size else (lambda t: None if t is None else t.double())
    batch, H, n, P = x.shape
    G, N = B.shape[1], B.shape[3]
    R = H // G
    ok = live_rows(lengths, batch, n, x.device)
    keep = ok[:, None, :, None]
    x = torch.where(keep, f(x), 0.0)
    b, c = (torch.where(keep, f(t), 0.0).repeat_interleave(R, 1) for t in (B, C))
    decay = torch.exp(torch.where(ok[:, None], dt * A.double()[:, None], 0.0))
    dt = torch.where(ok[:, None], dt.abs() if size else dt, 0.0)
    slope_ = torch.where(ok[:, None], slope_, 0.0)
    D = torch.zeros(H, dtype=torch.float64, device=x.device) if D is None else f(D)
    zero = torch.zeros(batch, H, N, P, dtype=torch.float64, device=x.device)
    h = zero if state is None else f(state)
    hs, y = [h], torch.zeros_like(x)
    for t in range(n):
        h = decay[:, :, t, None, None] * h + (dt[:, :, t, None] * b[:, :, t])[..., None] * x[:, :, t, None]
        hs.append(h)
        y[:, :, t] = (c[:, :, t, :, None] * h).sum(2) + D[:, None] * x[:, :, t]
    r = {"y": torch.where(keep, y, 0.0), "state": h}
    if dy is None:
        return r
    dy = torch.where(keep, f(dy), 0.0)
    g = zero if dstate is None else f(dstate)
    dx, dbh, dch = torch.zeros_like(x), torch.zeros_like(b), torch.zeros_like(c)
    da, v, w = (torch.zeros_like(dt) for _ in range(3))
    for t in reversed(range(n)):
        g = g + c[:, :, t, :, None] * dy[:, :, t, None]
        dch[:, :, t] = (hs[t + 1] * dy[:, :, t, None]).sum(-1)
        gb = (g * b[:, :, t, :, None]).sum(2)
        dx[:, :, t] = dt[:, :, t, None] * gb + D[:, None] * dy[:, :, t]
        dbh[:, :, t] = dt[:, :, t, None] * (g * x[:, :, t, None]).sum(-1)
        v[:, :, t] = (gb * x[:, :, t]).sum(-1)
        w[:, :, t] = (c[:, :, t] * dch[:, :, t]).sum(-1)
        g = decay[:, :, t, None, None] * g
        da[:, :, t] = (g * hs[t]).sum((-1, -2))
    if size:  # sums over the chunk instead of what they cancel to
        pad = -n % 128
        s = torch.nn.functional.pad(w + dt * v, (0, pad)).unflatten(-1, (-1, 128)).sum(-1).repeat_interleave(128, -1)[..., :n]
        da = da + s
    ddt = (A.double().abs() if size else A.double())[:, None] * da + v
    ddt = ddt * slope_
    r |= {"dx": dx, "d_dt": ddt, "dA": (da * dt).sum((0, 2)), "dB": dbh.unflatten(1, (G, R)).sum(2),
          "dC": dch.unflatten(1, (G, R)).sum(2), "dD": (dy * x).sum((0, 2, 3)), "d_dt_bias": ddt.sum((0, 2)), "d_state_in": g}
    return r


# names of outputs in which tensor-core operands are rounded to bf16 (twice at most: a weight or a
# state, and the weighted input that meets it)
ROUNDED = {"y", "dx", "dB", "dC"}


def ssm(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, state=None, lengths=None, dy=None, dstate=None,
        tensor_cores=False):
    """Dict of name -> (value, bound before the store's rounding)."""
    steps, sl = _steps(dt, dt_bias, dt_softplus)
    args = (x, steps, sl, A, B, C, D, state, lengths, dy, dstate)
    val, size = _scan(*args, False), _scan(*args, True)
    n, P, N = x.shape[2], x.shape[3], B.shape[3]
    nc = -(-n // 32)
    k = (1024 + N + P + 16 * nc + x.shape[0] * nc) * U
    top = lambda t: 1.0 if t is None else 1.0 + float(torch.where(torch.isfinite(t.double()), t.double(), 0.0).abs().max()) if t.numel() else 1.0  # noqa: E731
    under = 2.0 ** -126 * n * (n + 1) * N * P
    for t in (x, B, C, D, A, steps, state, dy, dstate):
        under *= top(t)
    out = {}
    for name, v in val.items():
        e = k * size[name] + under
        if tensor_cores and name in ROUNDED:
            e = e + 2.0 ** -7 * size[name]
        out[name] = (v, e)
    return out


# ------------------------------------------------------------------ norm
def norm(x, weight=None, bias=None, groups=1, eps=1e-5, center=True, gate=None, gate_first=False, kind="none", lengths=None,
         dy=None):
    B, n, d = x.shape
    m = d // groups
    ok = live_rows(lengths, B, n, x.device)[..., None]
    x = torch.where(ok, x.double(), 0.0)
    w = torch.ones(d, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(d, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    z_ = None if gate is None else torch.where(ok, gate.double(), 0.0)
    u = x * act(z_, "silu") if gate_first else x
    e_u = u.abs() * (e_sig(z_) + 4 * U) if gate_first else torch.zeros_like(u)
    by = lambda t: t.unflatten(-1, (groups, m))  # noqa: E731
    ug, eg = by(u), by(e_u)
    mean = ug.mean(-1, keepdim=True) if center else torch.zeros_like(ug[..., :1])
    e_mean = eg.mean(-1, keepdim=True) + (m + 4) * U * ug.abs().mean(-1, keepdim=True) if center else 0.0
    c = ug - mean
    e_c = eg + e_mean + 2 * U * c.abs()
    var = (c * c).mean(-1, keepdim=True)
    rs = 1 / (var + eps).sqrt()
    rel = ((c.abs() * e_c).mean(-1, keepdim=True) * rs * rs + (m + 16) * U)  # relative error of rs
    z = c * rs
    e_z = e_c * rs + z.abs() * rel
    zf, ezf = z.flatten(-2), e_z.flatten(-2)
    v, e_v = zf * w + b, ezf * w.abs() + 3 * U * ((zf * w).abs() + b.abs())
    after = gate is not None and not gate_first
    if after:
        y, e_y = v * act(z_, "silu"), e_v * act(z_, "silu").abs() + (v * act(z_, "silu")).abs() * (e_sig(z_) + 4 * U)
    elif gate is None and kind == "silu":
        y, e_y = act(v, "silu"), 1.1 * e_v + act(v, "silu").abs() * (e_sig(v) + 4 * U)
    else:
        y, e_y = v, e_v
    z0 = lambda t: torch.where(ok, t, 0.0)  # noqa: E731
    r = {"y": (z0(y), z0(e_y))}
    if dy is None:
        return r
    g = z0(dy.double())
    if after:
        sl, sg = slope(z_, "silu"), act(z_, "silu")
        e_sl = (1 + z_.abs()) * (e_sig(z_) + 4 * U)
        r["d_gate"] = (g * v * sl, g.abs() * (e_v * sl.abs() + v.abs() * e_sl + 4 * U * (v * sl).abs()))
        dv, e_dv = g * sg, (g * sg).abs() * (e_sig(z_) + 4 * U)
    elif gate is None and kind == "silu":
        dv = g * slope(v, "silu")
        e_dv = g.abs() * (0.6 * e_v + (1 + v.abs()) * (e_sig(v) + 4 * U))
    else:
        dv, e_dv = g, torch.zeros_like(g)
    k = (B * n / 8 + 64) * U
    r["d_weight"] = ((dv * zf).sum((0, 1)), (e_dv * zf.abs() + dv.abs() * ezf + k * (dv * zf).abs()).sum((0, 1)))
    r["d_bias"] = (dv.sum((0, 1)), (e_dv + k * dv.abs()).sum((0, 1)))
    q, e_q = by(dv * w), by(e_dv * w.abs() + 2 * U * (dv * w).abs())
    c1, a1 = (q * z).mean(-1, keepdim=True), (q * z).abs().mean(-1, keepdim=True)
    e_c1 = (e_q * z.abs() + q.abs() * e_z).mean(-1, keepdim=True) + (m + 4) * U * a1
    du = q - z * c1
    e_du = e_q + e_z * c1.abs() + z.abs() * e_c1 + 4 * U * (q.abs() + (z * c1).abs())
    if center:
        c0 = q.mean(-1, keepdim=True)
        du = du - c0
        e_du = e_du + e_q.mean(-1, keepdim=True) + (m + 8) * U * q.abs().mean(-1, keepdim=True)
    e_du = (e_du * rs + (du * rs).abs() * (rel + 2 * U)).flatten(-2)
    du = (du * rs).flatten(-2)
    if gate_first:
        sl, sg = slope(z_, "silu"), act(z_, "silu")
        r["d_gate"] = (du * x * sl, x.abs() * (e_du * sl.abs() + du.abs() * (1 + z_.abs()) * (e_sig(z_) + 4 * U)) + 4 * U * (du * x * sl).abs())
        du, e_du = du * sg, e_du * sg.abs() + (du * sg).abs() * (e_sig(z_) + 4 * U)
    r["dx"] = (z0(du), z0(e_du))
    if "d_gate" in r:
        r["d_gate"] = tuple(z0(t) for t in r["d_gate"])
    return r
