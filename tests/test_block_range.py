"""The norms around a block and the gated feed-forward block where values, plans or rings leave what
small batches of normal numbers reach.  Bounds as in test_block_operators.py."""

import math

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe
from tests import test_block_operators as ops
from tests.test_block_operators import _ffn_inputs, _gen, _rows

pytestmark = pytest.mark.gpu


# ------------------------------------------------------ plans that only large sizes take
WIDE = (2310, 1032, 2056)  # every product in tiles of 256 columns, with odd ends of M, N and K


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8])
def test_gated_ffn_in_wide_tiles(bits, dtype):
    """All elements of the outputs and gradients, as of small batches."""
    kind, limit = ("silu", 1.0) if bits == 8 else ("gelu", math.inf)
    ops.test_gated_ffn_saved(*WIDE, kind, limit, dtype)
    ops.test_gated_ffn_backward(*WIDE, kind, limit, bits, dtype)
    if bits == 16:
        ops.test_gated_ffn(*WIDE, kind, limit, dtype)


@pytest.mark.parametrize("M,H,I", [(8200, 264, 264), (300, 264, 4112), (2310, 1032, 2056)])
def test_a_corner_tile_of_many_steps(M, H, I):
    """A tile whose rows and columns one SM of the pair has alone, with many more K steps than stages:
    no wait runs out, and repeated calls give the same bits."""
    x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
    dout = _rows(_gen(M), M, H, torch.bfloat16)
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
    ws = torch.empty(q.qmoe_gated_ffn_backward_workspace_size(M, H, I), dtype=torch.uint8,
                     device="cuda")
    want = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, workspace=ws)
    out = q.qmoe_gated_ffn(x, w13, w2)
    for _ in range(50):
        got = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, workspace=ws)
        assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(out, q.qmoe_gated_ffn(x, w13, w2))
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)
