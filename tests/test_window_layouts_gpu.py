"""Windowed attention gives the same bits in every layout of one path: the tensor cores (bf16
rows of 16 bytes) and the CUDA cores add in different orders, so equal bits show that a layout
runs where the contiguous one runs.  Strides of dimensions with one element are never used."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def values(*shapes):
    gen = torch.Generator(device="cuda").manual_seed(7)
    return [torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in shapes]


def odd(t, stride):
    """The same elements with another stride wherever a dimension has one element."""
    return t.as_strided(t.shape, [stride if n == 1 else s for n, s in zip(t.shape, t.stride())])


@pytest.mark.parametrize("stride", [0, 1, 13])
@pytest.mark.parametrize("B,H,Hkv,n,nk", [(1, 1, 1, 300, 300), (1, 4, 2, 200, 200), (3, 2, 1, 150, 150), (2, 3, 1, 1, 200),
                                          (1, 1, 1, 1, 1)])
def test_strides_of_dimensions_with_one_element(B, H, Hkv, n, nk, stride):
    d, W, S = 64, 40, 3
    q, k, v, do = values((B, H, n, d), (B, Hkv, nk, d), (B, Hkv, nk, d), (B, H, n, d))
    o, lse = hla.window_forward(q, k, v, W, S, return_lse=True)
    want = hla.window_backward(q, k, v, o, lse, do, W, S)
    q1, k1, v1, do1, o1 = (odd(t, stride) for t in (q, k, v, do, o))
    out = odd(torch.zeros_like(o), stride)
    assert torch.equal(hla.window_forward(q1, k1, v1, W, S, out=out), o)
    outs = tuple(odd(torch.zeros_like(t), stride) for t in (q, k, v))
    for a, b in zip(hla.window_backward(q1, k1, v1, o1, lse, do1, W, S, out=outs), want):
        assert torch.equal(a, b)
    hla.hla_sync_status()


@pytest.mark.parametrize("stride", [0, 1, 13])
@pytest.mark.parametrize("B,H,Hkv,W,S", [(1, 4, 1, 300, 4), (1, 8, 2, 200, 0), (2, 4, 1, 130, 2), (1, 1, 1, 1, 0)])
def test_step_strides_of_dimensions_with_one_element(B, H, Hkv, W, S, stride):
    d = 64
    q, k, v, kc, vc = values((B, H, d), (B, Hkv, d), (B, Hkv, d), (B, Hkv, W + S, d), (B, Hkv, W + S, d))
    pos = torch.tensor([3 * (W + S) + 1, W + S - 1], device="cuda")[:B]
    kc1, vc1 = odd(kc.clone(), stride), odd(vc.clone(), stride)
    o = hla.window_step(kc, vc, pos, q, k, v, W, S)
    o1 = hla.window_step(kc1, vc1, pos, odd(q, stride), odd(k, stride), odd(v, stride), W, S)
    assert torch.equal(o, o1) and torch.equal(kc, kc1) and torch.equal(vc, vc1)
    hla.hla_sync_status()


@pytest.mark.parametrize("layout", ["tokens_first", "packed", "padded", "expanded"])
def test_layouts_with_wide_rows(layout):
    B, H, Hkv, n, d, W, S = 2, 4, 2, 300, 64, 50, 3
    q, k, v, do = values((B, H, n, d), (B, Hkv, n, d), (B, Hkv, n, d), (B, H, n, d))
    if layout == "expanded":
        k, v = k[:1].expand(B, Hkv, n, d), v[:1].expand(B, Hkv, n, d)
    o, lse = hla.window_forward(q, k.contiguous(), v.contiguous(), W, S, return_lse=True)
    want = hla.window_backward(q, k.contiguous(), v.contiguous(), o, lse, do, W, S)
    q1, k1, v1 = q, k, v
    if layout == "tokens_first":
        q1, k1, v1 = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    elif layout == "packed":
        pack = torch.cat([t.transpose(1, 2).reshape(B, n, -1) for t in (q, k, v)], -1)
        q1, k1, v1 = (x.unflatten(2, (-1, d)).transpose(1, 2) for x in pack.split([H * d, Hkv * d, Hkv * d], -1))
    elif layout == "padded":
        q1, k1, v1 = (torch.nn.functional.pad(t, (0, 8))[..., :d] for t in (q, k, v))
    o1, lse1 = hla.window_forward(q1, k1, v1, W, S, return_lse=True)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    for a, b in zip(hla.window_backward(q1, k1, v1, o1, lse1, do, W, S), want):
        assert torch.equal(a, b)
    hla.hla_sync_status()
