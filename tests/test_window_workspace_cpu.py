"""The backward's workspace stays in proportion to its gradients however many first tokens
there are: row sums, and beside a bounded part at most two fp32 copies of dk and dv."""
import pytest

import causal_prefix_scan_gb300 as hla
from causal_prefix_scan_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_F32])
@pytest.mark.parametrize("B,H,Hkv", [(1, 1, 1), (1, 32, 8), (8, 8, 8), (64, 16, 16)])
@pytest.mark.parametrize("n,window", [(1000, 30), (32768, 512), (32768, 16), (131072, 4096)])
@pytest.mark.parametrize("sinks", [0, 1, 64, 129, 1024, 2 ** 31 - 1])
def test_backward_workspace(B, H, Hkv, n, window, sinks, dtype):
    d = 128
    p = hla.hla_window_params(B, H, Hkv, n, n, d, d, dtype, window, sinks, 0.1, None)
    need = hla.hla_window_backward_workspace_size(p)
    rows, tile = B * H * n * 4, 128 * 2 * d * 4  # the largest tile: 128 keys of dk and dv
    assert rows <= need <= rows + 256 + 2 * B * Hkv * min(sinks, n + 127) * 2 * d * 4 + (2048 + 2 * B * Hkv) * tile
