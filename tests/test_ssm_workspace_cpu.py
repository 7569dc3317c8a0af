"""What the selective state space scan asks for as a workspace, next to the tensors that it is for."""
import ctypes

import pytest

import causal_prefix_scan_gb300 as hla
from causal_prefix_scan_gb300 import _build

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hla.library()


def size(lib, B, H, n, P, N, backward, dtype=hla.HLA_BF16):
    p = hla.hla_ssm_params(B, H, 1, n, P, N, dtype, 0, 256, None, None, None)
    return lib.hla_ssm_workspace_size(ctypes.byref(p), backward)


@pytest.mark.parametrize("dtype,width", [(hla.HLA_BF16, 2), (hla.HLA_F32, 4)])
@pytest.mark.parametrize("B,H,n,P,N", [(1, 64, 16384, 64, 128), (8, 64, 32768, 64, 128), (2, 32, 8192, 128, 128), (1, 1, 1 << 20, 64, 64), (512, 64, 600, 64, 64)])
def test_a_prompt_takes_less_than_its_tensors(lib, B, H, n, P, N, dtype, width):
    """Half of x, and spans of 64 MB (or of 2,048 states, or one of each head) with the states between them."""
    spans = max(64 * MB, 2048 * 4 * P * N, 4 * B * H * P * N) + 4 * B * H * P * N
    assert 0 < size(lib, B, H, n, P, N, 0, dtype) <= B * H * n * P * width // 2 + spans + 16 * MB


@pytest.mark.parametrize("B,H,n,P,N", [(2, 32, 8192, 64, 128), (8, 64, 32768, 64, 128), (1, 1, 1 << 20, 64, 64), (4, 8, 5000, 64, 40)])
def test_gradients_hold_the_states_once(lib, B, H, n, P, N):
    """bf16: on the tensor cores 32 KB and two images of a state for each chunk of 128 tokens, and 76 bytes a token
    and head; on the CUDA cores a state for 64 tokens, and the gradients of a span."""
    image = 128 * (64 if N <= 64 else 128)
    tc = B * H * -(-n // 128) * (32768 + 2 * image + 128 * 80)
    simt = B * H * -(-n // 64) * 4 * P * N + 64 * MB + 4 * B * H * P * N + 2 * 8 * B * n * N
    assert 0 < size(lib, B, H, n, P, N, 1) <= max(tc, simt) * 1.05 + 16 * MB


def test_one_size_for_both_paths(lib):
    """... and for every length up to a span the bytes that the states of all chunks take."""
    need = size(lib, 1, 2, 10, 64, 64, 0)
    assert need >= 2 * 64 * 64 * 4
