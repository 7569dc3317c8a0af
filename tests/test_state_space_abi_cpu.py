"""Refusals of the selective state space layer's entry points, before any CUDA work, and their
64-bit forms against autograd."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref
from causal_prefix_scan_gb300 import _build

ARG, UNSUPPORTED = hla.HLA_ERR_ARG, hla.HLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hla.library()


def T(p=4096, sb=64000, sh=640, st=64):
    return ctypes.byref(V(p, sb, sh, st))


def V(p=4096, sb=64000, sh=640, st=64):
    return hla.hla_tensor(p, sb, sh, st)


def conv(**kw):
    base = dict(B=1, n=10, d=64, width=4, in_dtype=hla.HLA_BF16, activation=1, weight=256, bias=512, lengths=None)
    return ctypes.byref(hla.hla_conv_params(**{**base, **kw}))


def ssm(**kw):
    base = dict(B=1, H=2, G=1, n=10, P=64, N=64, in_dtype=hla.HLA_BF16, dt_softplus=1, A=256, D=512, dt_bias=768, lengths=None)
    return ctypes.byref(hla.hla_ssm_params(**{**base, **kw}))


def norm(**kw):
    base = dict(B=1, n=10, d=64, groups=2, in_dtype=hla.HLA_BF16, center=1, activation=1, gate_first=0, eps=1e-5, weight=256,
                bias=512, lengths=None)
    return ctypes.byref(hla.hla_norm_params(**{**base, **kw}))


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), ARG), (dict(n=-1), ARG), (dict(d=0), ARG), (dict(in_dtype=5), ARG), (dict(activation=2), ARG), (dict(width=0), ARG),
    (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(n=2147483647), ARG), (dict(B=1 << 20, n=1 << 20, d=1 << 16), ARG)])
def test_conv_params(lib, kw, status):
    p = conv(**kw)
    assert lib.hla_conv_forward(p, T(), T(8192), None, None, None) == status
    assert lib.hla_conv_backward(p, T(), T(8192), T(12288), None, None, 4, 8, None, 256, 1 << 40, None) == status
    assert lib.hla_conv_step(p, T(), T(8192), 64, None) == status
    assert lib.hla_conv_backward_workspace_size(p) == 0
    assert hla.hla_last_error()


def test_conv_arguments(lib):
    fwd = lambda x=T(), y=T(8192), si=None, so=None, p=conv(): lib.hla_conv_forward(p, x, y, si, so, None)  # noqa: E731
    assert lib.hla_conv_forward(None, T(), T(8192), None, None, None) == ARG
    assert fwd(x=None) == ARG and fwd(y=None) == ARG and fwd(x=T(0)) == ARG and fwd(y=T()) == ARG
    assert fwd(x=T(4097)) == ARG and fwd(x=T(st=-1)) == ARG and fwd(y=T(8192, st=63)) == ARG
    assert fwd(si=64, so=64) == ARG and fwd(si=3) == ARG and fwd(so=5) == ARG
    assert fwd(p=conv(weight=None)) == ARG and fwd(p=conv(weight=2)) == ARG and fwd(p=conv(bias=6)) == ARG
    need = lib.hla_conv_backward_workspace_size(conv())
    assert need > 0 and need % 256 == 0

    def bwd(x=T(), dy=T(8192), dx=T(12288), si=None, do=None, dw=4, db=8, di=None, ws=256, n=need):
        return lib.hla_conv_backward(conv(), x, dy, dx, si, do, dw, db, di, ws, n, None)
    assert bwd(x=None) == ARG and bwd(dy=None) == ARG and bwd(dx=None) == ARG and bwd(dx=T()) == ARG and bwd(dx=T(8192)) == ARG
    assert bwd(dw=None) == ARG and bwd(dw=2) == ARG and bwd(db=1) == ARG and bwd(do=64, di=64) == ARG and bwd(si=64, di=64) == ARG
    assert bwd(ws=None) == ARG and bwd(n=need - 1) == ARG and bwd(ws=128) == ARG
    one = conv(n=1)
    assert lib.hla_conv_step(conv(), T(), T(8192), 64, None) == ARG
    assert lib.hla_conv_step(one, T(), T(8192), None, None) == ARG and lib.hla_conv_step(one, T(), T(8192), 3, None) == ARG
    assert lib.hla_conv_step(one, T(), T(), 64, None) == ARG and lib.hla_conv_step(one, T(), T(8192), 4096, None) == ARG


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), ARG), (dict(H=0), ARG), (dict(G=0), ARG), (dict(H=3, G=2), ARG), (dict(n=-1), ARG), (dict(P=0), ARG), (dict(N=0), ARG),
    (dict(in_dtype=2), ARG), (dict(P=129), UNSUPPORTED), (dict(N=200), UNSUPPORTED), (dict(n=2147483647), ARG),
    (dict(B=1 << 16, H=1 << 10), ARG)])
def test_ssm_params(lib, kw, status):
    p = ssm(**kw)
    x, dt, b, c, y = T(4096), T(8192), T(12288), T(16384), T(20480)
    g = hla.hla_ssm_gradients(V(24576), V(28672, 64000, 64, 1), V(32768), V(36864), 4, 8, 12, None)
    assert lib.hla_ssm_forward(p, x, dt, b, c, y, None, None, 256, 1 << 40, None) == status
    assert lib.hla_ssm_backward(p, x, dt, b, c, y, None, None, ctypes.byref(g), 256, 1 << 40, None) == status
    assert lib.hla_ssm_step(p, x, dt, b, c, y, 64, None) == status
    assert lib.hla_ssm_workspace_size(p, 0) == 0 and lib.hla_ssm_workspace_size(p, 1) == 0


def test_ssm_arguments(lib):
    t = dict(x=T(4096), dt=T(8192), b=T(12288), c=T(16384), y=T(20480))
    need = lib.hla_ssm_workspace_size(ssm(), 0)
    assert need > 0

    def fwd(p=ssm(), si=None, so=None, ws=256, n=need, **kw):
        a = {**t, **kw}
        return lib.hla_ssm_forward(p, a["x"], a["dt"], a["b"], a["c"], a["y"], si, so, ws, n, None)
    for name in t:
        assert fwd(**{name: None}) == ARG and fwd(**{name: T(0)}) == ARG and fwd(**{name: T(4097)}) == ARG
        assert fwd(**{name: T(4096, sb=-1)}) == ARG
    for name in ("x", "dt", "b", "c"):
        assert fwd(**{name: T(20480)}) == ARG
    assert fwd(y=T(20480, st=63)) == ARG and fwd(si=64, so=64) == ARG and fwd(si=2) == ARG
    assert fwd(ws=None) == ARG and fwd(n=need - 1) == ARG and fwd(ws=128) == ARG
    for kw in (dict(A=None), dict(A=3), dict(D=2), dict(dt_bias=1), dict(dt_softplus=0)):
        assert fwd(p=ssm(**kw)) == ARG
    need = lib.hla_ssm_workspace_size(ssm(), 1)
    outs = dict(dx=V(24576), d_dt=V(28672, 64000, 64, 1), db=V(32768), dc=V(36864), dA=4, dD=8, d_dt_bias=12, d_state_in=None)

    def bwd(p=ssm(), si=None, do=None, ws=256, n=need, **kw):
        g = hla.hla_ssm_gradients(**{**outs, **kw})
        return lib.hla_ssm_backward(p, t["x"], t["dt"], t["b"], t["c"], t["y"], si, do, ctypes.byref(g), ws, n, None)
    assert lib.hla_ssm_backward(ssm(), t["x"], t["dt"], t["b"], t["c"], t["y"], None, None, None, 256, need, None) == ARG
    for name in ("dx", "d_dt", "db", "dc"):
        assert bwd(**{name: V(0)}) == ARG and bwd(**{name: V(4096)}) == ARG
    assert bwd(db=V(24576)) == ARG and bwd(dx=V(24576, st=60)) == ARG and bwd(d_dt=V(28672, 64000, 9, 1)) == ARG
    assert bwd(dA=None) == ARG and bwd(dA=2) == ARG and bwd(dD=2) == ARG and bwd(d_dt_bias=2) == ARG and bwd(d_state_in=2) == ARG
    assert bwd(p=ssm(D=None)) == ARG and bwd(p=ssm(dt_bias=None)) == ARG
    assert bwd(do=64, d_state_in=64) == ARG and bwd(si=64, d_state_in=64) == ARG
    assert bwd(ws=None) == ARG and bwd(n=need - 1) == ARG and bwd(ws=128) == ARG
    step = lambda p=ssm(n=1), state=64, **kw: lib.hla_ssm_step(p, *({**t, **kw}[k] for k in t), state, None)  # noqa: E731
    assert step(p=ssm()) == ARG and step(state=None) == ARG and step(state=2) == ARG and step(state=4096) == ARG
    assert step(y=T(4096)) == ARG and step(state=20480) == ARG and step(dt=None) == ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(n=-1), dict(d=0), dict(groups=0), dict(groups=3), dict(in_dtype=2), dict(activation=7),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(weight=2), dict(bias=1), dict(n=2147483647)])
def test_norm_params(lib, kw):
    p = norm(**kw)
    assert lib.hla_norm_forward(p, T(), T(8192), T(12288), None) == ARG
    assert lib.hla_norm_backward(p, T(), T(8192), T(12288), T(16384), T(20480), 4, 8, 256, 1 << 40, None) == ARG
    assert lib.hla_norm_backward_workspace_size(p) == 0


def test_norm_arguments(lib):
    fwd = lambda x=T(), z=T(8192), y=T(12288), p=norm(): lib.hla_norm_forward(p, x, z, y, None)  # noqa: E731
    assert lib.hla_norm_forward(None, T(), None, T(8192), None) == ARG
    assert fwd(x=None) == ARG and fwd(y=None) == ARG and fwd(z=T(0)) == ARG and fwd(y=T()) == ARG and fwd(y=T(8192)) == ARG
    assert fwd(x=T(4097)) == ARG and fwd(y=T(12288, st=60)) == ARG
    assert fwd(z=None, p=norm(gate_first=1)) == ARG and fwd(p=norm(activation=0)) == ARG
    need = lib.hla_norm_backward_workspace_size(norm())
    assert need > 0 and need == lib.hla_norm_backward_workspace_size(norm(groups=64))

    def bwd(x=T(), z=T(8192), dy=T(12288), dx=T(16384), dz=T(20480), dw=4, db=8, ws=256, n=need):
        return lib.hla_norm_backward(norm(), x, z, dy, dx, dz, dw, db, ws, n, None)
    assert bwd(x=None) == ARG and bwd(dy=None) == ARG and bwd(dx=None) == ARG and bwd(dz=None) == ARG and bwd(z=None) == ARG
    assert bwd(dx=T()) == ARG and bwd(dz=T(12288)) == ARG and bwd(dz=T(16384)) == ARG and bwd(dw=2) == ARG and bwd(db=6) == ARG
    assert bwd(ws=None) == ARG and bwd(n=need - 1) == ARG and bwd(ws=128) == ARG


def calls():
    x, w, row = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(2, 8)
    h, b, dt, A = torch.zeros(2, 4, 5, 8), torch.zeros(2, 2, 5, 8), torch.zeros(2, 4, 5), torch.zeros(4)
    return {
        "conv_forward": lambda s: hla.conv_forward(x, w, stream=s),
        "conv_workspace": lambda s: hla.conv_workspace(x, w, stream=s),
        "conv_backward": lambda s: hla.conv_backward(x, x, w, stream=s),
        "conv_step": lambda s: hla.conv_step(torch.zeros(2, 3, 8), row, w, stream=s),
        "ssm_workspace": lambda s: hla.ssm_workspace(h, b, stream=s),
        "ssm_forward": lambda s: hla.ssm_forward(h, dt, A, b, b, stream=s),
        "ssm_backward": lambda s: hla.ssm_backward(h, dt, A, b, b, h, stream=s),
        "ssm_step": lambda s: hla.ssm_step(torch.zeros(2, 4, 8, 8), h[:, :, 0], dt[:, :, 0], A, b[:, :, 0], b[:, :, 0], stream=s),
        "norm_forward": lambda s: hla.norm_forward(x, stream=s),
        "norm_workspace": lambda s: hla.norm_workspace(x, stream=s),
        "norm_backward": lambda s: hla.norm_backward(x, x, stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_stream_of_another_device(lib, name, monkeypatch):
    monkeypatch.setattr(hla, "_current", lambda t: t.device)  # CPU tensors stand in for those of the current device
    stream = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        calls()[name](stream)


def test_tensor_arguments(lib, monkeypatch):
    monkeypatch.setattr(hla, "_current", lambda t: t.device)
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    for bad in (lambda: hla.conv_forward(x[0], w), lambda: hla.conv_forward(x, w[:4]), lambda: hla.conv_forward(x, w, activation="gelu"),
                lambda: hla.conv_forward(x, w, state_in=torch.zeros(2, 4, 8)), lambda: hla.conv_step(torch.zeros(2, 2, 8), x[:, 0], w),
                lambda: hla.conv_forward(x.transpose(1, 2), torch.zeros(5, 4)), lambda: hla.norm_forward(x[0]),
                lambda: hla.norm_forward(x, gate=x[:1]), lambda: hla.norm_forward(x, weight=w[:, 0][:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        hla.conv_forward(x, w.double())
    h, b, dt, A = torch.zeros(2, 4, 5, 8), torch.zeros(2, 2, 5, 6), torch.zeros(2, 4, 5), torch.zeros(4)
    for bad in (lambda: hla.ssm_forward(h[0], dt, A, b, b), lambda: hla.ssm_forward(h, dt[:1], A, b, b), lambda: hla.ssm_forward(h, dt, A[:2], b, b),
                lambda: hla.ssm_forward(h, dt, A, b, b[..., :5]), lambda: hla.ssm_forward(h, dt, A, b[0], b[0]),
                lambda: hla.ssm_forward(h, dt, A, b, b, state_in=torch.zeros(2, 4, 8, 6)),
                lambda: hla.ssm_step(torch.zeros(2, 4, 8, 6), h[:, :, 0], dt[:, :, 0], A, b[:, :, 0], b[:, :, 0])):
        with pytest.raises(ValueError):
            bad()


def leaves(gen, **shapes):
    return {k: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_() for k, s in shapes.items()}


def compare(got, want):
    for name, w in want.items():
        assert torch.allclose(got[name][0], w, atol=1e-11), name


@pytest.mark.parametrize("kind", ["none", "silu"])
def test_the_convolutions_form_has_autograds_gradient(kind):
    gen = torch.Generator().manual_seed(0)
    t = leaves(gen, x=(2, 7, 3), w=(3, 4), b=(3,), st=(2, 3, 3))
    L, dy, ds = torch.tensor([7, 2]), torch.randn(2, 7, 3, dtype=torch.float64), torch.randn(2, 3, 3, dtype=torch.float64)
    out = 0.0
    for s in range(2):
        n = int(L[s])
        xs = torch.cat([t["st"][s], t["x"][s, :n]])
        y = ref.act(t["b"] + sum(xs[i:i + n] * t["w"][:, i] for i in range(4)), kind)
        out = out + (y * dy[s, :n]).sum() + (xs[n:] * ds[s]).sum()
    out.backward()
    d = {k: v.detach() for k, v in t.items()}
    got = ref.conv(d["x"], d["w"], d["b"], kind, d["st"], L, dy, ds)
    compare(got, {"dx": t["x"].grad, "d_weight": t["w"].grad, "d_bias": t["b"].grad, "d_state_in": t["st"].grad})


@pytest.mark.parametrize("softplus", [False, True])
def test_the_scans_form_has_autograds_gradient(softplus):
    gen = torch.Generator().manual_seed(0)
    t = leaves(gen, x=(2, 4, 6, 3), dt=(2, 4, 6), A=(4,), B=(2, 2, 6, 5), C=(2, 2, 6, 5), D=(4,), bias=(4,), st=(2, 4, 5, 3))
    L, dy, ds = torch.tensor([6, 4]), torch.randn(2, 4, 6, 3, dtype=torch.float64), torch.randn(2, 4, 5, 3, dtype=torch.float64)
    h, out = t["st"], 0.0
    for i in range(6):
        live = (i < L)[:, None]
        dt = t["dt"][:, :, i]
        dt = torch.nn.functional.softplus(dt + t["bias"]) if softplus else dt
        b, c = (t[k][:, :, i].repeat_interleave(2, 1) for k in "BC")
        new = torch.exp(dt * t["A"])[..., None, None] * h + (dt[..., None] * b)[..., None] * t["x"][:, :, i, None]
        h = torch.where(live[..., None, None], new, h)
        y = (c[..., None] * h).sum(2) + t["D"][:, None] * t["x"][:, :, i]
        out = out + torch.where(live[..., None], y * dy[:, :, i], 0.0).sum()
    (out + (h * ds).sum()).backward()
    d = {k: v.detach() for k, v in t.items()}
    got = ref.ssm(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"] if softplus else None, softplus, d["st"], L, dy, ds)
    want = {"dx": t["x"].grad, "d_dt": t["dt"].grad, "dA": t["A"].grad, "dB": t["B"].grad, "dC": t["C"].grad, "dD": t["D"].grad,
            "d_state_in": t["st"].grad}
    compare(got, {**want, **({"d_dt_bias": t["bias"].grad} if softplus else {})})
    assert torch.allclose(got["state"][0], h.detach())


@pytest.mark.parametrize("gate,first,kind", [(False, False, "none"), (False, False, "silu"), (True, False, "silu"), (True, True, "silu")])
@pytest.mark.parametrize("center", [False, True])
def test_the_norms_form_has_autograds_gradient(gate, first, kind, center):
    gen = torch.Generator().manual_seed(0)
    t = leaves(gen, x=(2, 3, 8), w=(8,), b=(8,), z=(2, 3, 8))
    L, dy = torch.tensor([3, 1]), torch.randn(2, 3, 8, dtype=torch.float64)
    u = t["x"] * ref.act(t["z"], "silu") if first else t["x"]
    u = u.unflatten(-1, (2, 4))
    if center:
        u = u - u.mean(-1, keepdim=True)
    v = (u / ((u * u).mean(-1, keepdim=True) + 0.1).sqrt()).flatten(-2) * t["w"] + t["b"]
    y = v * ref.act(t["z"], "silu") if gate and not first else ref.act(v, kind) if not gate else v
    keep = (torch.arange(3) < L[:, None])[..., None]
    torch.where(keep, y * dy, 0.0).sum().backward()
    d = {k: v.detach() for k, v in t.items()}
    got = ref.norm(d["x"], d["w"], d["b"], 2, 0.1, center, d["z"] if gate else None, first, kind, L, dy)
    compare(got, {"dx": t["x"].grad, "d_weight": t["w"].grad, "d_bias": t["b"].grad, **({"d_gate": t["z"].grad} if gate else {})})
