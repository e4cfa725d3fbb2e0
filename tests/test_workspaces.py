"""A workspace's size is what its tensor holds: expanded tensors, whose elements share bytes, are refused."""
import os

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_gather_gb300")


@pytest.fixture(scope="module")
def bq():
    if not os.path.exists(os.path.join(PKG, "libbq.so")):
        import __graft_entry__
        __graft_entry__.build()
    import block_quantized_moe_gather_gb300 as m
    return m


def test_bytes_of_a_workspace(bq):
    torch = pytest.importorskip("torch")
    ws = torch.empty(64, dtype=torch.uint8)
    assert bq._workspace("w", ws) == (ws.data_ptr(), 64) and bq._workspace("w", None) == (None, 0)
    assert bq._workspace("w", torch.empty(8, 4))[1] == 128
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1, 8).expand(64, 8), ws[::2]):
        with pytest.raises(bq.BQError, match="the workspace has shape"):
            bq._workspace("w", bad)


@pytest.mark.gpu
def test_expanded_workspaces_are_refused(lib):
    import torch
    new = (lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda"))
    small = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24)
    h, rows = 64, [new(4, 64) for _ in range(6)]
    logits, ids = new(4, 16), new(4, 2, dtype=torch.int32)
    calls = [lambda: lib.residual_norm_backward(*rows, gain=new(h), dgain=new(h), workspace=small),
             lambda: lib.moe_balance_loss(logits, ids, new(1, 16, dtype=torch.int32), new(1, 16), new(2), small),
             lambda: lib.moe_route_backward(logits, ids, new(4, 2), new(4, 16), dbias=new(16), workspace=small)]
    for call in calls:
        before = lib.launch_count()
        with pytest.raises(lib.BQError, match="the workspace has shape"):
            call()
        assert lib.launch_count() == before
