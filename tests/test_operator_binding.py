"""The operators' Python binding: what becomes of errors that kernels find."""

import gc

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

gpu = pytest.mark.gpu


def _lora(M, ids):
    K, N, R, L = 64, 48, 8, 3
    t = torch.ones
    kw = dict(device="cuda", dtype=torch.bfloat16)
    return q.qmoe_lora_linear(t(M, K, **kw), t(N, K, **kw), t(L, R, K, **kw), t(L, N, R, **kw),
                              ids, torch.ones(L, device="cuda"))


@gpu
def test_errors_of_calls_without_a_workspace():
    ok, bad_id = (qmoe.QMOE_OK, 0), (qmoe.QMOE_ERR_BAD_ID, qmoe.QMOE_FLAG_BAD_ID)
    x = torch.randn(4, 64, device="cuda")
    good = torch.tensor([[0, 7], [3, 1], [-1, 2], [2, 5]], dtype=torch.int32, device="cuda")
    bad = good.clone()
    bad[1, 1] = 8
    for M in (4, 20):
        ids = torch.arange(M, dtype=torch.int32, device="cuda") % 3
        q.moe_sort_tokens(x, good, 8)
        _lora(M, ids)
        assert q.qmoe_default_read_error() == ok
        q.moe_sort_tokens(x, bad, 8)
        _lora(M, ids)  # another operator's call does not hide it
        assert q.qmoe_default_read_error() == bad_id
        # nor do calls that bring a workspace, have no tokens or are refused
        ws = torch.empty(q.qmoe_sort_workspace_size(4, 2, 8), dtype=torch.uint8, device="cuda")
        q.moe_sort_tokens(x, good, 8, workspace=ws)
        assert q.qmoe_default_read_error() == bad_id
        q.moe_sort_tokens(x, good, 8)
        assert q.qmoe_default_read_error() == ok
        ids[2] = 3
        _lora(M, ids)
        assert q.qmoe_default_read_error() == bad_id
        _lora(M, ids.clamp(max=2))
        assert q.qmoe_default_read_error() == ok
    q.moe_sort_tokens(x[:0], good[:0], 8)
    assert q.qmoe_default_read_error() == ok
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.moe_sort_tokens(x, bad, 8, stream=side)
    assert q.qmoe_default_read_error(side) == bad_id
    q.moe_sort_tokens(x, good, 8)
    torch.cuda.synchronize()


@gpu
def test_kept_workspaces_do_not_grow():
    x = torch.randn(4096, 8, device="cuda")
    ids = torch.zeros(4096, 2, dtype=torch.int32, device="cuda")
    q.moe_sort_tokens(x, ids, 8)
    gc.collect()
    before = torch.cuda.memory_allocated()
    for _ in range(5):
        q.moe_sort_tokens(x, ids, 8)
    assert torch.cuda.memory_allocated() == before
