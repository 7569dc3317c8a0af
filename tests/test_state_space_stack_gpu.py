"""The selective state space layer as it is used: convolution, scan and gated norm together, for
prompts, single tokens and training, on streams and in graphs."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import state_space_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
H, G, P, N, W = 4, 2, 64, 64, 4
DI, DC = H * P, H * P + 2 * G * N


class Layer:
    """z, xBC and dt as a projection gives them; everything behind it."""

    def __init__(self, dtype, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.gen, self.dtype, self.r = gen, dtype, r
        self.w, self.b, self.A, self.D, self.bias = r(DC, W) / 2, 0.1 * r(DC), -torch.rand(H, generator=gen, device="cuda") - 0.5, r(H), r(H) - 2
        self.nw, self.nb = 1 + 0.1 * r(DI), 0.1 * r(DI)

    def inputs(self, B, n):
        return tuple(self.r(B, n, d).to(self.dtype) for d in (DI, DC, H))

    @staticmethod
    def split(u):
        f = lambda a, h, w: u[..., a:a + h * w].unflatten(-1, (h, w)).transpose(1, 2)  # noqa: E731
        return f(0, H, P), f(DI, G, N), f(DI + G * N, G, N)

    def ssm_kw(self):
        return dict(D=self.D, dt_bias=self.bias, dt_softplus=True)

    def norm_kw(self, z):
        return dict(groups=G, gate=z, activation="silu")

    def prompt(self, z, xbc, dt, lengths=None, stream=None):
        u, cs = hla.conv_forward(xbc, self.w, self.b, "silu", return_state=True, lengths=lengths, stream=stream)
        x, B, C = self.split(u)
        y, hs = hla.ssm_forward(x, dt.transpose(1, 2), self.A, B, C, return_state=True, lengths=lengths, stream=stream, **self.ssm_kw())
        y = y.transpose(1, 2).flatten(2)
        o = hla.norm_forward(y, self.nw, self.nb, lengths=lengths, stream=stream, **self.norm_kw(z))
        return o, cs, hs, u, y

    def step(self, cs, hs, z, xbc, dt, live=None):
        u = hla.conv_step(cs, xbc, self.w, self.b, "silu", lengths=live)
        x, B, C = (t[:, :, 0] for t in self.split(u[:, None]))
        y = hla.ssm_step(hs, x, dt, self.A, B, C, lengths=live, **self.ssm_kw())
        return hla.norm_forward(y.flatten(1)[:, None], self.nw, self.nb, **self.norm_kw(z[:, None]))[:, 0]

    def gradients(self, z, xbc, dt, do, lengths=None, stream=None):
        o, _, _, u, y = self.prompt(z, xbc, dt, lengths, stream)
        n = hla.norm_backward(y, do, self.nw, self.nb, lengths=lengths, stream=stream, **self.norm_kw(z))
        x, B, C = self.split(u)
        du = torch.zeros_like(u)
        dx, dB, dC = self.split(du)
        ddt = torch.zeros_like(dt)
        s = hla.ssm_backward(x, dt.transpose(1, 2), self.A, B, C, n.dx.unflatten(-1, (H, P)).transpose(1, 2), lengths=lengths,
                             out=(dx, ddt.transpose(1, 2), dB, dC), stream=stream, **self.ssm_kw())
        c = hla.conv_backward(xbc, du, self.w, self.b, "silu", lengths=lengths, stream=stream)
        return dict(o=o, z=n.d_gate, xbc=c.dx, dt=ddt, A=s.dA, D=s.dD, bias=s.d_dt_bias, w=c.d_weight, b=c.d_bias, nw=n.d_weight, nb=n.d_bias)

    def plain(self, z, xbc, dt, do):
        """The same layer in 64 bits by autograd."""
        leaf = {k: v.double().detach().requires_grad_() for k, v in dict(z=z, xbc=xbc, dt=dt, A=self.A, D=self.D, bias=self.bias, w=self.w,
                                                                       b=self.b, nw=self.nw, nb=self.nb).items()}
        Bn, n = z.shape[:2]
        xs = torch.nn.functional.pad(leaf["xbc"], (0, 0, W - 1, 0))
        u = ref.act(leaf["b"] + sum(xs[:, i:i + n] * leaf["w"][:, i] for i in range(W)), "silu")
        x, B, C = self.split(u)
        steps = torch.nn.functional.softplus(leaf["dt"] + leaf["bias"], threshold=60.0).transpose(1, 2)
        h = torch.zeros(Bn, H, N, P, dtype=torch.float64, device="cuda")
        ys = []
        for t in range(n):
            b, c = (v[:, :, t].repeat_interleave(H // G, 1) for v in (B, C))
            h = torch.exp(steps[:, :, t] * leaf["A"])[..., None, None] * h + (steps[:, :, t, None] * b)[..., None] * x[:, :, t, None]
            ys.append((c[..., None] * h).sum(2) + leaf["D"][:, None] * x[:, :, t])
        y = torch.stack(ys, 1).flatten(2).unflatten(-1, (G, -1))
        y = y - y.mean(-1, keepdim=True)
        y = (y / ((y * y).mean(-1, keepdim=True) + 1e-5).sqrt()).flatten(-2) * leaf["nw"] + leaf["nb"]
        o = y * ref.act(leaf["z"], "silu")
        (o * do.double()).sum().backward()
        return dict(o=o.detach(), **{k: v.grad for k, v in leaf.items()})


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


# In 2-norms: fp32 carries a few hundred roundings of 2^-24 through three operators; bf16 stores u, y
# and each gradient between the operators once and rounds the scan's weights and states once: about
# ten independent roundings of at most 2^-9 on the way, which the norm and the activations scale by
# less than 4.
@pytest.mark.parametrize("dtype,tol", [(F32, 1e-4), (BF16, 10 * 4 * 2.0 ** -9)])
@pytest.mark.parametrize("n", [1, 5, 200])
def test_training_step(n, dtype, tol):
    m = Layer(dtype)
    z, xbc, dt = m.inputs(2, n)
    do = m.r(2, n, DI).to(dtype)
    got, want = m.gradients(z, xbc, dt, do), m.plain(z, xbc, dt, do)
    hla.hla_sync_status()
    for k in want:
        if n == 1 and k in ("A",):  # the state before the only token is zero: no gradient
            assert float(got[k].abs().max()) <= 1e-6
            continue
        assert rel(got[k], want[k]) <= tol, k


@pytest.mark.parametrize("dtype,tol", [(F32, 1e-4), (BF16, 10 * 4 * 2.0 ** -9)])
def test_prompt_then_tokens(dtype, tol):
    m = Layer(dtype, 1)
    z, xbc, dt = m.inputs(3, 150)
    whole = m.prompt(z, xbc, dt)[0]
    o, cs, hs, _, _ = m.prompt(z[:, :140], xbc[:, :140], dt[:, :140])
    outs = [o] + [m.step(cs, hs, z[:, t], xbc[:, t], dt[:, t])[:, None] for t in range(140, 150)]
    assert rel(torch.cat(outs, 1), whole.double()) <= tol


def test_ragged_prompts_then_tokens():
    """Each sequence of a padded batch goes on from its own length as it would alone."""
    m = Layer(F32, 2)
    z, xbc, dt = m.inputs(3, 150)
    L = torch.tensor([150, 1, 77], dtype=torch.int32, device="cuda")
    nz, nx, nd = m.inputs(3, 1)
    o, cs, hs, _, _ = m.prompt(z, xbc, dt, L)
    live = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
    kept = cs[2].clone(), hs[2].clone()
    s = m.step(cs, hs, nz[:, 0], nx[:, 0], nd[:, 0], live)
    assert torch.equal(cs[2], kept[0]) and torch.equal(hs[2], kept[1])
    for b in (0, 1):
        k = int(L[b])
        t = [torch.cat([a[b:b + 1, :k], c[b:b + 1]], 1) for a, c in ((z, nz), (xbc, nx), (dt, nd))]
        alone = m.prompt(*t)[0]
        assert rel(o[b, :k], alone[0, :k].double()) <= 1e-5 and rel(s[b], alone[0, k].double()) <= 1e-4


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_another_stream(how):
    m = Layer(BF16, 3)
    z, xbc, dt = m.inputs(2, 200)
    do = m.r(2, 200, DI).to(BF16)
    want = m.gradients(z, xbc, dt, do)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):  # (the zeroed gradients of the test itself)
        got = m.gradients(z, xbc, dt, do, stream=st if how == "stream" else st.cuda_stream)
    st.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_captured_and_replayed():
    m = Layer(BF16, 4)
    z, xbc, dt = m.inputs(2, 200)
    do = m.r(2, 200, DI).to(BF16)
    m.gradients(z, xbc, dt, do)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.gradients(z, xbc, dt, do)
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (z, xbc, dt, do):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        want = m.gradients(z, xbc, dt, do)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_two_graphs_on_one_workspace():
    m = Layer(BF16, 7)
    _, xbc, dt = m.inputs(2, 300)
    x, B, C = m.split(xbc)
    ws = hla.ssm_workspace(x, B, backward=True)
    call = lambda s: hla.ssm_backward(x, dt.transpose(1, 2), m.A, B, C, x, workspace=ws, **{**m.ssm_kw(), "D": m.D * s})  # noqa: E731
    want = [call(s) for s in (1.0, 2.0)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in (1.0, 2.0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(s))
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, r) if a is not None)


def test_calls_at_once_on_two_streams():
    m = Layer(BF16, 8)
    sets = [m.inputs(1, 600) for _ in range(2)]
    dos = [m.r(1, 600, DI).to(BF16) for _ in range(2)]
    want = [m.gradients(*s, d) for s, d in zip(sets, dos)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, d, st in zip(sets, dos, streams):
        with torch.cuda.stream(st):
            got.append(m.gradients(*s, d))
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert all(torch.equal(w[k], r[k]) for k in w)
