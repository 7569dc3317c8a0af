"""Refusals of the gated recurrence's and the windowed attention's entry points, before any
CUDA work, and their 64-bit forms against autograd."""
import ctypes

import pytest
import torch

import causal_prefix_scan_gb300 as hla
import constant_state_ref as ref
from causal_prefix_scan_gb300 import _build

ARG, UNSUPPORTED = hla.HLA_ERR_ARG, hla.HLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hla.library()


def T(p=4096, sb=640, sh=64, st=64):
    return ctypes.byref(hla.hla_tensor(p, sb, sh, st))


def gp(**kw):
    base = dict(B=1, n=10, d=64, in_dtype=hla.HLA_BF16, gate=hla.HLA_GATE_GIVEN, rate=None, lengths=None)
    return hla.hla_gated_params(**{**base, **kw})


def wp(**kw):
    base = dict(B=1, H=1, Hkv=1, n=10, nk=10, d=64, dv=64, in_dtype=hla.HLA_BF16, window=4, sinks=1, scale=0.1, lengths=None)
    return hla.hla_window_params(**{**base, **kw})


@pytest.mark.parametrize("kw", [dict(B=0), dict(n=-1), dict(d=0), dict(in_dtype=5), dict(gate=3), dict(gate=-1),
                                dict(gate=hla.HLA_GATE_RATE), dict(B=1 << 30, n=1 << 30), dict(n=2147483647)])
def test_gated_params(lib, kw):
    p = gp(**kw)
    b = ctypes.byref(p)
    assert lib.hla_gated_forward(b, T(), T(8192), T(12288), None, None, None, 0, None) == ARG
    assert lib.hla_gated_backward(b, T(), T(8192), T(12288), T(16384), None, None, T(20480), T(24576), None, None, None, 0, None) == ARG
    assert lib.hla_gated_step(b, T(), T(8192), T(12288), 4, 4, None) == ARG
    assert lib.hla_gated_workspace_size(b) == 0
    assert hla.hla_last_error()


def test_gated_arguments(lib):
    b = ctypes.byref(gp())
    x, g, y = T(4096), T(8192), T(12288)
    fwd = lambda x, g, y, si=None, so=None, ws=None, n=0, p=b: lib.hla_gated_forward(p, x, g, y, si, so, ws, n, None)  # noqa: E731
    assert lib.hla_gated_forward(None, x, g, y, None, None, None, 0, None) == ARG
    assert fwd(None, g, y) == ARG and fwd(x, None, y) == ARG and fwd(x, g, None) == ARG and fwd(T(0), g, y) == ARG
    assert fwd(x, g, T(4096)) == ARG                        # y is x
    assert fwd(T(4097), g, y) == ARG                        # half an element
    assert fwd(T(st=-64), g, y) == ARG and fwd(T(sb=-1), g, y) == ARG
    assert fwd(x, g, T(12288, st=32)) == ARG                # rows of y overlap
    assert fwd(x, g, T(12288, sb=0), p=ctypes.byref(gp(B=2))) == ARG
    assert fwd(x, g, y, 4, 4) == ARG                        # state_out is state_in
    assert fwd(x, g, y, 2, None) == ARG                     # misaligned state
    long = ctypes.byref(gp(n=1000))
    assert fwd(x, g, T(12288, sb=64000), p=long) == ARG     # needs a workspace
    need = lib.hla_gated_workspace_size(long)
    assert need > 0
    assert fwd(x, g, T(12288, sb=64000), ws=256, n=need - 1, p=long) == ARG
    assert fwd(x, g, T(12288, sb=64000), ws=128, n=need, p=long) == ARG  # misaligned workspace
    step = ctypes.byref(gp(n=1))
    assert lib.hla_gated_step(b, x, g, y, 4, 4, None) == ARG            # not one token
    assert lib.hla_gated_step(step, x, g, y, None, 4, None) == ARG and lib.hla_gated_step(step, x, g, y, 4, None, None) == ARG
    bwd = lambda x, g, y, dy, dx, dg, dr=None, do=None, di=None: lib.hla_gated_backward(  # noqa: E731
        b, x, g, y, dy, None, do, dx, dg, dr, di, None, 0, None)
    dy, dx, dg = T(16384), T(20480), T(24576)
    assert bwd(x, g, None, dy, dx, dg) == ARG and bwd(x, g, y, dy, dx, None) == ARG
    assert bwd(x, g, y, dy, T(16384), dg) == ARG and bwd(x, g, y, dy, dx, T(20480)) == ARG
    assert bwd(x, g, y, dy, dx, dg, dr=4) == ARG                        # no rates with this gate
    assert bwd(x, g, y, dy, dx, dg, do=4, di=4) == ARG


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), ARG), (dict(H=0), ARG), (dict(Hkv=0), ARG), (dict(H=3, Hkv=2), ARG), (dict(d=0), ARG), (dict(dv=0), ARG),
    (dict(in_dtype=2), ARG), (dict(window=0), ARG), (dict(sinks=-1), ARG), (dict(scale=float("inf")), ARG),
    (dict(scale=float("nan")), ARG), (dict(n=-1), ARG), (dict(nk=9), ARG), (dict(d=129), UNSUPPORTED),
    (dict(dv=200), UNSUPPORTED), (dict(nk=2147483647), ARG), (dict(B=1 << 30, H=4, Hkv=4), ARG)])
def test_window_params(lib, kw, status):
    b = ctypes.byref(wp(**kw))
    q, k, v, o = T(4096), T(8192), T(12288), T(16384)
    assert lib.hla_window_forward(b, q, k, v, o, None, None) == status
    assert lib.hla_window_backward(b, q, k, v, o, 4, T(20480), T(24576), T(28672), T(32768), 256, 1 << 40, None) == status
    assert lib.hla_window_backward_workspace_size(b) == 0
    if not {"n", "nk"} & set(kw):
        s = ctypes.byref(wp(**{**kw, "n": 1}))
        assert lib.hla_window_step(s, q, k, v, T(20480), T(24576), 8, o, None) == status
        assert lib.hla_window_cache_fill(s, k, v, T(20480), T(24576), None) == status


def test_window_arguments(lib):
    b = ctypes.byref(wp())
    q, k, v, o = T(4096), T(8192), T(12288), T(16384)
    fwd = lambda q, k, v, o, lse=None: lib.hla_window_forward(b, q, k, v, o, lse, None)  # noqa: E731
    assert fwd(None, k, v, o) == ARG and fwd(q, None, v, o) == ARG and fwd(q, k, None, o) == ARG and fwd(q, k, v, None) == ARG
    assert fwd(q, k, v, T(4096)) == ARG and fwd(q, k, v, o, 2) == ARG and fwd(T(4097), k, v, o) == ARG
    assert fwd(q, k, v, T(16384, st=63)) == ARG and fwd(T(sh=-1), k, v, o) == ARG
    go, dq, dk, dv = T(20480), T(24576), T(28672), T(32768)
    need = lib.hla_window_backward_workspace_size(b)
    assert need > 0
    bwd = lambda lse=4, dq=dq, dk=dk, dv=dv, ws=256, n=need: lib.hla_window_backward(b, q, k, v, o, lse, go, dq, dk, dv, ws, n, None)  # noqa: E731
    assert bwd(lse=None) == ARG and bwd(dq=T(4096)) == ARG and bwd(dk=T(24576)) == ARG and bwd(dv=None) == ARG
    assert bwd(ws=None) == ARG and bwd(n=need - 1) == ARG and bwd(ws=128) == ARG
    none = ctypes.byref(wp(n=0))
    assert lib.hla_window_backward(none, q, k, v, o, 4, go, dq, dk, dv, 256, need, None) == ARG
    s = ctypes.byref(wp(n=1))
    kc, vc = T(20480), T(24576)
    step = lambda q=q, k=k, v=v, kc=kc, vc=vc, pos=8, o=o, p=s: lib.hla_window_step(p, q, k, v, kc, vc, pos, o, None)  # noqa: E731
    assert step(p=b) == ARG and step(q=None) == ARG and step(pos=None) == ARG and step(pos=4) == ARG
    assert step(vc=T(20480)) == ARG and step(kc=T(8192)) == ARG and step(o=T(4096)) == ARG
    assert step(kc=T(20480, st=0)) == ARG                               # slots overlap
    assert step(p=ctypes.byref(wp(n=1, window=2147483647, sinks=5))) == ARG
    assert step(p=ctypes.byref(wp(n=1, window=2147483640, sinks=0))) == ARG  # counters of slots would overflow
    fill = lambda k=k, v=v, kc=kc, vc=vc: lib.hla_window_cache_fill(b, k, v, kc, vc, None)  # noqa: E731
    assert fill(k=None) == ARG and fill(vc=None) == ARG and fill(kc=T(8192)) == ARG and fill(vc=T(20480)) == ARG


@pytest.mark.parametrize("gate", ["given", "sigmoid", "rate"])
def test_the_recurrence_form_has_autograds_gradient(gate):
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, n, d = 2, 9, 5
    x, g, st = r(B, n, d).requires_grad_(), torch.sigmoid(r(B, n, d)).requires_grad_(), r(B, d).requires_grad_()
    rate = torch.rand(d, generator=gen, dtype=torch.float64).add(0.1).requires_grad_()
    L, dy, ds = torch.tensor([9, 4]), r(B, n, d), r(B, d)
    h, ys = st, []
    for t in range(n):
        a, f = ref.gates(gate, g[:, t], rate)
        live = (t < L)[:, None]
        h = torch.where(live, a * h + f * x[:, t], h)
        ys.append(torch.where(live, h, 0.0))
    y = torch.stack(ys, 1)
    ((y * dy).sum() + (h * ds).sum()).backward()
    a = [t.detach() for t in (x, g, st, rate)]
    ry, rs, _, _ = ref.gated_forward(a[0], a[1], gate, a[3], a[2], L)
    assert torch.allclose(ry, y) and torch.allclose(rs, h)
    got = ref.gated_backward(a[0], a[1], ry, dy, gate, a[3], a[2], ds, L)
    for name, want in (("dx", x.grad), ("dg", g.grad), ("d_state_in", st.grad)) + ((("d_rate", rate.grad),) if gate == "rate" else ()):
        assert torch.allclose(got[name][0], want, atol=1e-12), name


def test_the_attention_form_has_autograds_gradient():
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k, v = r(2, 4, 7, 6).requires_grad_(), r(2, 2, 11, 6).requires_grad_(), r(2, 2, 11, 5).requires_grad_()
    L, do = torch.tensor([11, 7]), r(2, 4, 7, 5)
    o, lse, _, _ = ref.window_forward(q, k, v, 3, 2, 0.4, L)
    (o * do).sum().backward()
    got = ref.window_backward(*(t.detach() for t in (q, k, v, o, lse)), do, 3, 2, 0.4, L)
    for name, want in (("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert torch.allclose(got[name][0], want, atol=1e-12), name
