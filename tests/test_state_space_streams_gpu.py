"""The selective state space layer's calls on a stream that is not the current one: what a call
allocates and clears, and its kernels, belong to the stream that it is given."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla

pytestmark = pytest.mark.gpu
ENTRIES = ("hla_conv_forward", "hla_conv_backward", "hla_conv_step", "hla_ssm_forward", "hla_ssm_backward", "hla_ssm_step",
           "hla_norm_forward", "hla_norm_backward")


def calls(B=2, n=100):
    z = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    x, w, cs, L = z(B, n, 8), z(8, 4), z(B, 3, 8), torch.tensor([n] + [3] * (B - 1), dtype=torch.int32, device="cuda")
    h, b, dt, A, hs = z(B, 4, n, 8), z(B, 2, n, 8), z(B, 4, n), -z(4), z(B, 4, 8, 8)
    return {
        "hla_conv_forward": lambda s: hla.conv_forward(x, w, lengths=L, return_state=True, stream=s),
        "hla_conv_backward": lambda s: hla.conv_backward(x, x, w, lengths=L, want_dstate=True, stream=s),
        "hla_conv_step": lambda s: hla.conv_step(cs, x[:, 0], w, lengths=L, stream=s),
        "hla_ssm_forward": lambda s: hla.ssm_forward(h, dt, A, b, b, lengths=L, return_state=True, stream=s),
        "hla_ssm_backward": lambda s: hla.ssm_backward(h, dt, A, b, b, h, lengths=L, want_dstate=True, stream=s),
        "hla_ssm_step": lambda s: hla.ssm_step(hs, h[:, :, 0], dt[:, :, 0], A, b[:, :, 0], b[:, :, 0], lengths=L, stream=s),
        "hla_norm_forward": lambda s: hla.norm_forward(x, lengths=L, stream=s),
        "hla_norm_backward": lambda s: hla.norm_backward(x, x, x[0, 0], lengths=L, stream=s),
    }


@pytest.mark.parametrize("given", ["default handle", "default", "side handle", "side"])
@pytest.mark.parametrize("entry", ENTRIES)
def test_the_stream_of_a_call(entry, given, monkeypatch):
    stream = torch.cuda.default_stream() if given.startswith("default") else torch.cuda.Stream()
    seen = []
    monkeypatch.setattr(hla, entry, lambda *a: seen.append((torch.cuda.current_stream().cuda_stream, hla._stream(a[-1]))))
    with torch.cuda.stream(torch.cuda.Stream()):  # neither of the two
        calls()[entry](stream.cuda_stream if given.endswith("handle") else stream)
    assert seen == [(stream.cuda_stream, stream.cuda_stream)]
    torch.cuda.synchronize()


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("entry", ENTRIES)
def test_padded_batches_on_the_default_stream_by_its_handle(entry):
    """New outputs are cleared ahead of the kernels, on their stream."""
    n = 1 if entry.endswith("step") else 3000
    want = flat(calls(16, n)[entry](None))  # (a step changes its state: a new one each time)
    torch.cuda.synchronize()
    for _ in range(5):
        call = calls(16, n)[entry]
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            got = flat(call(0))
            torch.cuda.synchronize()
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    hla.hla_sync_status()
