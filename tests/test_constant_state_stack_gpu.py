"""The constant-state layers together, as a stack uses them: a gated recurrence whose
output rows hold q, k and v, windowed attention on views of those rows, masked HLA behind
it; a padded prompt, then token by token on the three states, captured into one graph; and
the gradient back through the two new layers."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla
import constant_state_ref as ref
from gpu_helpers import TOL_BF16

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
B, H, Hkv, n, more, d, W, S = 3, 4, 2, 200, 40, 64, 48, 4
WIDTH = (H + 2 * Hkv) * d


def heads(y):
    """q, k, v views of rows [B, n, WIDTH] (or of [B, WIDTH])."""
    q, k, v = (t.unflatten(-1, (-1, d)) for t in y.split([H * d, Hkv * d, Hkv * d], -1))
    return (q, k, v) if y.dim() == 2 else tuple(t.transpose(1, 2) for t in (q, k, v))


def inputs():
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    return r(B, n + more, WIDTH), r(B, n + more, WIDTH), torch.rand(WIDTH, generator=gen, device="cuda") + 0.05


def test_prompt_then_captured_steps():
    x, g, rate = inputs()
    L = torch.tensor([n, 7, 0], dtype=torch.int32, device="cuda")
    # the prompt
    y, state = hla.gated_forward(x[:, :n], g[:, :n], "rate", rate, return_state=True, lengths=L)
    q, k, v = heads(y)
    kc, vc = hla.window_cache(B, Hkv, W, S, d)
    hla.window_cache_fill(kc, vc, k, v, W, S, lengths=L)
    o = hla.window_forward(q, k, v, W, S, lengths=L)
    # a third layer on the first sequence, whose prompt is whole
    qk = torch.nn.functional.normalize(o[:1].float(), dim=-1).to(BF16).contiguous()
    vals = o[:1].contiguous()
    o3, hstate = hla.forward(qk, qk, vals, chunk=64, return_state=True)
    rows = torch.arange(B, device="cuda")
    pos = L.long()
    xs, gs = torch.zeros(B, WIDTH, dtype=BF16, device="cuda"), torch.zeros(B, WIDTH, dtype=BF16, device="cuda")
    yt, ot = torch.zeros_like(xs), torch.zeros(B, H, d, dtype=BF16, device="cuda")
    o3t, qkt = torch.zeros(H, d, dtype=BF16, device="cuda"), torch.zeros(H, d, dtype=BF16, device="cuda")

    def step():
        hla.gated_step(state, xs, gs, "rate", rate, out=yt)
        hla.window_step(kc, vc, pos, *heads(yt), W, S, out=ot)
        qkt.copy_(torch.nn.functional.normalize(ot[0].float(), dim=-1))
        hla.decode_step(hstate, qkt, qkt, ot[0].contiguous(), H, out=o3t)
        pos.add_(1)

    keep = [t.clone() for t in (state, kc, vc, pos) + hstate.astuple()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, was in zip((state, kc, vc, pos) + hstate.astuple(), keep):
        t.copy_(was)
    ys, os_, o3s = [], [], []
    for _ in range(more):
        xs.copy_(x[rows, pos])
        gs.copy_(g[rows, pos])
        graph.replay()
        ys.append(yt.clone()), os_.append(ot.clone()), o3s.append(o3t.clone())
    hla.hla_sync_status()
    for b in range(B):
        m = int(L[b])
        ry, rs, Ey, Es = ref.gated_forward(x[b:b + 1, :m + more], g[b:b + 1, :m + more], "rate", rate)
        whole = torch.cat([y[b, :m], torch.stack([t[b] for t in ys])])[None]  # the rows as they were rounded
        ref.close(whole, ry, Ey, f"recurrence {b}")
        ref.close(state[b:b + 1], rs, Es, f"state {b}")
        ro, _, Eo, _ = ref.window_forward(*heads(whole), W, S, d ** -0.5, None, ref.half_step(BF16))
        got = torch.cat([o[b, :, :m], torch.stack([t[b] for t in os_], 1)], 1)[None]
        ref.close(got, ro, Eo, f"attention {b}")
        if b == 0:  # the third layer against one forward over all its tokens
            qk = torch.nn.functional.normalize(got.float(), dim=-1).to(BF16).contiguous()
            want = hla.forward(qk, qk, got.contiguous(), chunk=64)[0, :, m:].double()
            have = torch.stack(o3s, 1).double()
            assert float((have - want).norm() / want.norm()) <= TOL_BF16


def test_gradient_through_both_layers():
    x, g, rate = inputs()
    L = torch.tensor([n + more, 130, 1], dtype=torch.int32, device="cuda")
    y = hla.gated_forward(x, g, "rate", rate, lengths=L)
    q, k, v = heads(y)
    o, lse = hla.window_forward(q, k, v, W, S, lengths=L, return_lse=True)
    do = torch.randn(o.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    dy = torch.zeros_like(y)
    hla.window_backward(q, k, v, o, lse, do, W, S, lengths=L, out=heads(dy))
    want = ref.window_backward(q, k, v, o, lse, do, W, S, d ** -0.5, L, ref.half_step(BF16))
    for name, got in zip(("dq", "dk", "dv"), heads(dy)):
        ref.close(got, *want[name], name)
    r = hla.gated_backward(x, g, y, dy, "rate", rate, lengths=L)
    hla.hla_sync_status()
    want = ref.gated_backward(x, g, y, dy, "rate", rate, lengths=L)
    for name in ("dx", "dg", "d_rate"):
        ref.close(getattr(r, name), *want[name], name)
