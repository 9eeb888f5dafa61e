"""The gated block's calls with the error word apart from the workspace."""

import ctypes
import math

import pytest
import torch

from quantized_moe_grouped_route_gb300 import qmoe

P = ctypes.c_void_p
A = P(4096)  # never read: what follows is refused before anything is enqueued


@pytest.fixture(scope="module")
def lib():
    from quantized_moe_grouped_route_gb300 import build
    build.build()
    return qmoe.lib()


def _forward(lib, x, w13, w2, M, H, I, out, ws, n, error):
    return lib.qmoe_gated_ffn_error_at(x, 0, H, w13, w2, 0, math.inf, M, H, I, out, None, None, ws, n,
                                       error, None)


def _backward(lib, dout, x, w13, w2, kept, M, H, I, grads, ws, n, error):
    return lib.qmoe_gated_ffn_backward_error_at(dout, 0, H, x, H, None, w13, w2, kept, None, 0,
                                                math.inf, M, H, I, *grads, ws, n, error, None)


def test_refusals(lib):
    M, H, I = 4, 64, 128
    n = lib.qmoe_gated_ffn_workspace_size(M, H, I)
    m = lib.qmoe_gated_ffn_backward_workspace_size(M, H, I, 16)
    for error in (None, P(4097), P(4098)):
        assert _forward(lib, A, A, A, M, H, I, A, A, n, error) == qmoe.QMOE_ERR_ARG
        assert _backward(lib, A, A, A, A, A, M, H, I, (A, A, A), A, m, error) == qmoe.QMOE_ERR_ARG
    assert _forward(lib, A, A, A, M, H, I, A, A, n - 1, A) == qmoe.QMOE_ERR_WORKSPACE
    assert _backward(lib, A, A, A, A, A, M, H, I, (A, A, A), A, m - 1, A) == qmoe.QMOE_ERR_WORKSPACE
    assert _forward(lib, A, A, A, 0, H, I, A, A, n, None) == qmoe.QMOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_the_word_is_where_it_is_said_to_be(lib, M):
    """Cleared at error_dev; nothing around it and nothing of the workspace's first block is written."""
    H, I, dt = 128, 264, torch.bfloat16
    x, w13, w2 = (torch.randn(s, device="cuda", dtype=dt) for s in ((M, H), (2 * I, H), (H, I)))
    out, kept = torch.empty_like(x), torch.randn(M, 2 * I, device="cuda", dtype=dt)
    grads = [torch.empty_like(t) for t in (x, w13, w2)]
    words = torch.full((64,), 0x55, dtype=torch.int32, device="cuda")
    error = P(words.data_ptr() + 4 * 17)
    n = lib.qmoe_gated_ffn_workspace_size(M, H, I)
    m = lib.qmoe_gated_ffn_backward_workspace_size(M, H, I, 16)
    ws = torch.full((max(n, m),), 0xAB, dtype=torch.uint8, device="cuda")
    p = [P(t.data_ptr()) for t in (x, w13, w2, out, kept, ws)]
    torch.cuda.synchronize()
    for call in (lambda: _forward(lib, p[0], p[1], p[2], M, H, I, p[3], p[5], n, error),
                 lambda: _backward(lib, p[0], p[0], p[1], p[2], p[4], M, H, I,
                                   [P(t.data_ptr()) for t in grads], p[5], m, error)):
        words.fill_(0x55)
        torch.cuda.synchronize()
        assert call() == qmoe.QMOE_OK
        torch.cuda.synchronize()
        assert int(words[17]) == 0 and int((words == 0x55).sum()) == 63
        assert (ws[:256] == 0xAB).all()
