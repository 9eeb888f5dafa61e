"""Refusals of the norms' backward call that concern a full gate's gradient of the gate's own type (no
GPU needed)."""

import ctypes

import pytest

from quantized_moe_grouped_route_gb300 import qmoe

P = ctypes.c_void_p
A = P(4096)  # never read: what follows is refused before anything is enqueued
TOKEN, FULL, OWN = 0, 2, 16


@pytest.fixture(scope="module")
def lib():
    from quantized_moe_grouped_route_gb300 import build
    build.build()
    return qmoe.lib()


def test_own_gradient_refusals(lib):
    n = lib.qmoe_block_norm_backward_workspace_size(4, 8)

    def call(form, gate_type=2, dgate=A, size=n):
        return lib.qmoe_block_norm_backward(A, 8, None, 8, A, 0, 8, None, 8, 1.0, A, gate_type, form, 8,
                                            0, None, None, 0, 0.0, None, None, 4, 8, A, None, dgate,
                                            None, None, A, size, None)
    # of a full gate alone
    for form in (TOKEN + OWN, 1 + OWN, 3 + OWN, OWN - 1, 2 * OWN):
        assert call(form) == qmoe.QMOE_ERR_ARG
    # aligned as its own type
    assert call(FULL + OWN, dgate=P(4098)) == qmoe.QMOE_ERR_ARG
    for form, gate_type, dgate in ((FULL, 2, P(4098)), (FULL + OWN, 0, P(4098)), (FULL + OWN, 2, P(4100))):
        assert call(form, gate_type, dgate, n - 1) == qmoe.QMOE_ERR_WORKSPACE
