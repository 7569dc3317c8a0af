"""Plain 64-bit forms of the gated recurrence and of windowed attention, with bounds on
what rounding may do to a kernel's results.

Bounds.  u = 2^-24 is half a step of fp32, eps(t)/2 that of the element type.
  Recurrence: a gate and an input factor come out within K u of their values (the
  exponential's argument is off by half a step of up to 10, its result by two steps, the
  quotient by two), one token adds one rounding, so the error of the state obeys
      E_t <= |a_t| E_{t-1} + K u (|a_t| H_{t-1} + |b_t|),   H the same scan of absolute values,
  whatever the grouping of tokens into tiles (a product of gates carries the sum of its
  factors' relative errors).  K = 32.
  Attention: a score of width d is off by (d + 8) u scale sum |q||k|, a probability by that
  relatively (twice, with the maximum), sums of N terms by N u of their absolute sum; the
  tensor-core path rounds P and dS to bf16, half a step each.
"""
import torch

U = 2.0 ** -24
K_GATE = 32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gates(gate, g, rate):
    """a_t and the factor of x_t."""
    if gate == "given":
        return g, torch.ones_like(g)
    if gate == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(-g)
    u = rate * torch.sigmoid(g)
    return torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def gated_forward(x, g, gate, rate=None, state=None, lengths=None):
    """(y, state, bound of |y|'s error, bound of the state's) in 64 bits; rows behind a
    length are zero."""
    x, g = x.double(), g.double()
    rate = None if rate is None else rate.double()
    B, n, d = x.shape
    h = torch.zeros(B, d, dtype=torch.float64, device=x.device) if state is None else state.double().clone()
    H, E = h.abs(), torch.zeros_like(h)
    y, Ey = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(n):
        a, f = gates(gate, g[:, t], rate)
        b = f * x[:, t]
        live = torch.ones(B, 1, dtype=torch.bool, device=x.device) if lengths is None else (t < lengths)[:, None]
        E = torch.where(live, a.abs() * E + K_GATE * U * (a.abs() * H + b.abs()), E)
        H = torch.where(live, a.abs() * H + b.abs(), H)
        h = torch.where(live, a * h + b, h)
        y[:, t], Ey[:, t] = torch.where(live, h, 0.0), torch.where(live, E, 0.0)
    return y, h, Ey, E


def gated_backward(x, g, y, dy, gate, rate=None, state=None, d_state=None, lengths=None):
    """Gradients and bounds: a dict of name -> (value, bound before the store's rounding)."""
    x, g, y, dy = (t.double() for t in (x, g, y, dy))
    rate = None if rate is None else rate.double()
    B, n, d = x.shape
    zero = torch.zeros(B, d, dtype=torch.float64, device=x.device)
    h0 = zero if state is None else state.double()
    c = zero.clone() if d_state is None else d_state.double().clone()
    C, E = c.abs(), zero.clone()
    out = {k: (torch.zeros_like(x), torch.zeros_like(x)) for k in ("dx", "dg")}
    dr, Er = torch.zeros(d, dtype=torch.float64, device=x.device), torch.zeros(d, dtype=torch.float64, device=x.device)
    ku = K_GATE * U
    for t in reversed(range(n)):
        live = torch.ones(B, 1, dtype=torch.bool, device=x.device) if lengths is None else (t < lengths)[:, None]
        a, f = gates(gate, g[:, t], rate)
        prev = y[:, t - 1] if t else h0
        gh, G = dy[:, t] + c, dy[:, t].abs() + C
        Eg = E + ku * G  # of gh
        if gate == "given":
            dg, Edg = gh * prev, (Eg + ku * G) * prev.abs()
        elif gate == "sigmoid":
            dg, Edg = gh * (prev - x[:, t]) * a * f, (Eg + ku * G) * (prev.abs() + x[:, t].abs()) * a * f
        else:
            s = torch.sigmoid(g[:, t])
            du = gh * (x[:, t] * a * a / f - a * prev)
            Edu = (Eg + ku * G) * (x[:, t].abs() * a * a / f + a * prev.abs())
            dg, Edg = du * rate * s * (1 - s), Edu * rate * s * (1 - s)
            dr += torch.where(live, du * s, 0.0).sum(0)
            # 16 + 8 additions in a tile, then one per 8 tiles and sequence
            Er += torch.where(live, Edu * s * (1 + (64 + B * (n // 1024 + 1)) / K_GATE), 0.0).sum(0)
        for name, val, bound in (("dx", gh * f, f * (Eg + ku * G)), ("dg", dg, Edg)):
            out[name][0][:, t] = torch.where(live, val, 0.0)
            out[name][1][:, t] = torch.where(live, bound, 0.0)
        E = torch.where(live, a.abs() * (E + ku * G), E)
        C = torch.where(live, a.abs() * G, C)
        c = torch.where(live, a * gh, c)
    out["d_state_in"] = (c, E)
    if gate == "rate":
        out["d_rate"] = (dr, Er)
    return out


def mask(n, nk, window, sinks, device):
    """[n, nk]: query row i (position nk - n + i) sees key j."""
    p = torch.arange(nk - n, nk, device=device)[:, None]
    j = torch.arange(nk, device=device)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def _clean(x, lengths, p0=0):
    """Rows at positions from the length on as zeros: they may hold anything."""
    if lengths is None:
        return x
    ok = p0 + torch.arange(x.shape[2], device=x.device) < lengths[:, None]
    return torch.where(ok[:, None, :, None] if x.dim() == 4 else ok[:, None], x, torch.zeros((), dtype=x.dtype, device=x.device))


def window_scores(q, k, window, sinks, scale, lengths):
    n, nk, H = q.shape[2], k.shape[2], q.shape[1]
    q, k = _clean(q, lengths, nk - n).double(), _heads(_clean(k, lengths), H)
    see = mask(n, nk, window, sinks, q.device)[None, None]
    if lengths is not None:
        see = see & (torch.arange(nk - n, nk, device=q.device) < lengths[:, None])[:, None, :, None]
    s = (q @ k.transpose(-1, -2)) * scale
    # of a score, relative error of its probability
    delta = (q.shape[-1] + 8) * U * abs(scale) * (q.abs() @ k.abs().transpose(-1, -2))
    return torch.where(see, s, -torch.inf), torch.where(see, delta, 0.0), see


def window_forward(q, k, v, window, sinks, scale, lengths=None, rounded=0.0):
    """o, lse and the bounds of their errors before o's own rounding; `rounded`: half a step
    of the type that P is rounded to (0: kept in fp32)."""
    H, nk = q.shape[1], k.shape[2]
    s, delta, see = window_scores(q, k, window, sinks, scale, lengths)
    live = see.any(-1)
    v = _heads(_clean(v, lengths), H)
    lse = torch.where(live, torch.logsumexp(s, -1), 0.0)
    p = torch.where(see, torch.exp(s - lse[..., None]), 0.0)
    worst = delta.amax(-1, keepdim=True) + 8 * U
    o = p @ v
    return (o, lse, (p * (2 * delta + 2 * worst + 2 * rounded + 2 * nk * U)) @ v.abs(),
            torch.where(live, worst[..., 0] + nk * U + 4 * U * lse.abs(), 0.0))


def window_backward(q, k, v, o, lse, do, window, sinks, scale, lengths=None, rounded=0.0):
    """(value, bound before the store's rounding) of dq, dk, dv, from the given o and lse."""
    B, H, n, d = q.shape
    Hkv, nk = k.shape[1], k.shape[2]
    s, delta, see = window_scores(q, k, window, sinks, scale, lengths)
    p0 = nk - n
    qd, dod, od = (_clean(t, lengths, p0).double() for t in (q, do, o))
    lse = _clean(lse, lengths, p0).double()
    kd, vd = _heads(_clean(k, lengths), H), _heads(_clean(v, lengths), H)
    p = torch.where(see, torch.exp(s - lse[..., None]), 0.0)
    Ep = p * (2 * delta + 4 * U * (lse.abs()[..., None] + torch.where(see, s, 0.0).abs()) + 8 * U)
    dp = dod @ vd.transpose(-1, -2)
    D = (dod * od).sum(-1, keepdim=True)
    Edp = (v.shape[-1] + 8) * U * (dod.abs() @ vd.abs().transpose(-1, -2) + (dod * od).abs().sum(-1, keepdim=True))
    dS = p * (dp - D) * scale
    EdS = abs(scale) * (Ep * (dp.abs() + D.abs()) + p * Edp) + (rounded + 4 * U) * dS.abs()
    Ep = Ep + rounded * p
    fold = lambda x: x.view(B, Hkv, H // Hkv, nk, -1).sum(2)  # noqa: E731
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    N = 2 * n * (H // Hkv) * U
    return {"dq": (dS @ kd, (EdS + 2 * nk * U * dS.abs()) @ kd.abs()),
            "dk": (fold(T(dS) @ qd), fold(T(EdS + N * dS.abs()) @ qd.abs())),
            "dv": (fold(T(p) @ dod), fold(T(Ep + N * p) @ dod.abs()))}


def close(got, ref, bound, what):
    """|got - ref| within the bound and half a step of got's type, everywhere."""
    tol = bound * 1.001 + half_step(got.dtype) * (ref.abs() + bound) + 1e-37
    bad = ~((got.double() - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{float(got[i])} for {float(ref[i])}, tolerance {float(tol[i])}")
