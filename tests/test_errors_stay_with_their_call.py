"""An error of one call is that call's alone."""

import ctypes

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

P = ctypes.c_void_p


def _cudart():
    """The CUDA runtime that PyTorch has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libcudart" in line}
    if not paths:
        pytest.skip("no CUDA runtime library loaded")
    return ctypes.CDLL(sorted(paths)[0])


@pytest.mark.gpu
def test_a_call_after_one_that_failed():
    """A call into a stream whose capture has been spoiled (by a synchronisation, which a capture
    refuses) fails; the calls after it on another stream do not."""
    x = torch.randn(4, 64, device="cuda", dtype=torch.bfloat16)
    out, w = torch.empty_like(x), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    want = q.qmoe_checkpoint8(x)
    codes, scales = (torch.zeros_like(t) for t in want)
    back = torch.empty_like(x)
    packed = torch.randint(0, 256, (1, 128, 64), device="cuda", dtype=torch.uint8)
    factors = torch.full((1, 128, 8), 0x38, device="cuda", dtype=torch.uint8)
    repacked = [torch.empty(n, device="cuda", dtype=torch.uint8)
                for n in (qmoe.lib().qmoe_repacked_fp4_size(1, 128, 128),
                          qmoe.lib().qmoe_repacked_scale_size(1, 128, 128))]
    selftest = torch.empty(1 << 20, device="cuda", dtype=torch.int16)
    torch.cuda.synchronize()
    lib, cudart, stream = qmoe.lib(), _cudart(), torch.cuda.Stream()
    s = P(stream.cuda_stream)

    def norm():
        return lib.qmoe_block_norm(P(x.data_ptr()), 0, 64, None, 64, 1.0, None, 0, 0, 1, 0,
                                   P(w.data_ptr()), None, 0, 0.0, 1e-6, 4, 64, P(out.data_ptr()), None,
                                   None, None, s)
    for call in (lambda: lib.qmoe_checkpoint8(P(x.data_ptr()), 0, 64, 4, 64, P(codes.data_ptr()),
                                              P(scales.data_ptr()), None),
                 lambda: lib.qmoe_checkpoint8_restore(P(want[0].data_ptr()), P(want[1].data_ptr()), 0, 4,
                                                      64, P(back.data_ptr()), None),
                 lambda: lib.moe_nvfp4_repack(P(packed.data_ptr()), P(factors.data_ptr()), 1, 128, 128,
                                              qmoe.QMOE_W2, P(repacked[0].data_ptr()),
                                              P(repacked[1].data_ptr()), None),
                 lambda: lib.qmoe_selftest_dequant(P(selftest.data_ptr()), None)):
        assert cudart.cudaStreamBeginCapture(s, 2) == 0
        assert norm() == qmoe.QMOE_OK
        assert cudart.cudaStreamSynchronize(s) != 0
        assert norm() == qmoe.QMOE_ERR_CUDA
        graph = P()
        assert cudart.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0 and not graph.value
        cudart.cudaGetLastError()
        assert call() == qmoe.QMOE_OK
        torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert torch.equal(back, q.qmoe_checkpoint8_restore(*want))
