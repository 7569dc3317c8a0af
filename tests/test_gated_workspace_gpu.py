"""A workspace whose header is not ready is reported, and nothing is computed from it."""
import pytest
import torch

import causal_prefix_scan_gb300 as hla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float32, 33)])
@pytest.mark.parametrize("tickets,base", [(1000, 0), (0, 1000), (2 ** 62, 3), (5, 2 ** 62), (100, 0)])
def test_header_that_was_not_zeroed(tickets, base, dtype, d):
    n = 400
    x = torch.ones(1, n, d, dtype=dtype, device="cuda")
    ws = hla.gated_workspace(x)
    head = ws.view(torch.int64)  # tickets, and their count at the call's begin
    mark = [torch.full_like(x, 7.0) for _ in range(3)]
    y = hla.gated_forward(x, x)
    hla.hla_sync_status()
    for call in (lambda: hla.gated_forward(x, x, out=mark[0], workspace=ws),
                 lambda: hla.gated_backward(x, x, y, x, out=(mark[1], mark[2]), workspace=ws)):
        head[0], head[1] = tickets, base
        call()
        with pytest.raises(hla.HlaError, match="workspace") as e:
            hla.hla_sync_status()
        assert e.value.status == hla.HLA_ERR_ARG
        hla.hla_sync_status()  # reported once
    assert all(bool((m == 7).all()) for m in mark)
    ws.zero_()
    assert torch.equal(hla.gated_forward(x, x, workspace=ws), y)
    hla.hla_sync_status()
