"""What a call allocates and clears belongs to the stream that its kernels run on, however the
stream is given: the default stream's handle is 0."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla

pytestmark = pytest.mark.gpu
ENTRIES = ("hla_gated_forward", "hla_gated_backward", "hla_gated_step", "hla_window_forward", "hla_window_backward",
           "hla_window_cache_fill", "hla_window_step")


def calls():
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, row, L = z(2, 100, 8), z(2, 8), torch.tensor([100, 3], dtype=torch.int32, device="cuda")
    q, t, lse, pos, c = z(2, 2, 5, 8), z(2, 2, 8), z(2, 2, 5), torch.zeros(2, dtype=torch.int64, device="cuda"), z(2, 2, 4, 8)
    return {
        "hla_gated_forward": lambda s: hla.gated_forward(x, x, lengths=L, return_state=True, stream=s),
        "hla_gated_backward": lambda s: hla.gated_backward(x, x, x, x, lengths=L, stream=s),
        "hla_gated_step": lambda s: hla.gated_step(row.clone(), row, row, lengths=L, stream=s),
        "hla_window_forward": lambda s: hla.window_forward(q, q, q, 3, lengths=L, return_lse=True, stream=s),
        "hla_window_backward": lambda s: hla.window_backward(q, q, q, q, lse, q, 3, lengths=L, stream=s),
        "hla_window_cache_fill": lambda s: hla.window_cache_fill(c, c.clone(), q, q, 4, stream=s),
        "hla_window_step": lambda s: hla.window_step(c, c.clone(), pos, t, t, t, 4, stream=s),
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


def test_calls_on_the_default_stream_by_its_handle():
    """A padded batch, whose new outputs and workspace are cleared on the stream of the call."""
    n, d = 5000, 512
    x = torch.ones(4, n, d, device="cuda")
    L = torch.tensor([n, 1, 0, 70], dtype=torch.int32, device="cuda")
    want, state = hla.gated_forward(x, x, lengths=L, return_state=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(20):
            y, s = hla.gated_forward(x, x, lengths=L, return_state=True, stream=0)
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(s, state)
    hla.hla_sync_status()
