"""Calls of the C ABI from two host threads at once, each with a stream and a workspace of its
own and with a problem of another size: every call succeeds, with the results it has alone."""

import threading

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

pytestmark = pytest.mark.gpu
CALLS = 400


def _p(t):
    return qmoe._ptr(t)


def _lora(M, K, N, R, L):
    g = torch.Generator(device="cuda").manual_seed(M + R)
    x, w, a, b = (torch.randn(*s, generator=g, device="cuda").bfloat16()
                  for s in ((M, K), (N, K), (L, R, K), (L, N, R)))
    s = torch.ones(L, device="cuda")
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    n = q.qmoe_lora_workspace_size(M, K, N, R, L)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(stream):
        return qmoe.lib().qmoe_lora_linear(_p(x), 0, K, _p(w), _p(a), _p(b), _p(ids), _p(s), None,
                                           0, _p(out), M, K, N, R, L, _p(ws), n, stream)
    return call, [out]


def _sort(M, E, k):
    g = torch.Generator(device="cuda").manual_seed(M + E)
    x = torch.randn(M, 64, generator=g, device="cuda")
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    xs = torch.empty(M * k, 64, device="cuda")
    offs, sp, pp = (torch.empty(n, dtype=torch.int32, device="cuda")
                    for n in (E + 1, M * k, M * k))
    n = q.qmoe_sort_workspace_size(M, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(stream):
        return qmoe.lib().moe_sort_tokens(_p(x), 2, 64, _p(ids), M, 64, k, E, _p(xs), _p(offs),
                                          _p(sp), _p(pp), _p(ws), n, stream)
    return call, [xs, offs, sp, pp]


def _route(M, E, k):
    g = torch.Generator(device="cuda").manual_seed(M + E)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    offs, sp, pp = (torch.empty(n, dtype=torch.int32, device="cuda")
                    for n in (E + 1, M * k, M * k))
    tiles = torch.zeros(qmoe.qmoe_max_tiles(M, k, E, 64), 3, dtype=torch.int32, device="cuda")
    count = torch.empty(1, dtype=torch.int32, device="cuda")
    n = qmoe.qmoe_route_workspace_size(M, k, E, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(stream):
        return qmoe.lib().moe_route(_p(ids), M, k, E, 64, _p(offs), _p(sp), _p(pp), _p(tiles),
                                    _p(count), _p(ws), n, stream)
    return call, [offs, sp, pp, count]


PAIRS = {
    "adapter GEMM": lambda: (_lora(70, 256, 300, 16, 3), _lora(128, 256, 300, 128, 60)),
    "adapter x A^T": lambda: (_lora(600, 512, 128, 64, 4), _lora(257, 1024, 128, 64, 4)),
    "sort": lambda: (_sort(3000, 900, 2), _sort(2000, 2048, 2)),
    "route": lambda: (_route(500, 64, 2), _route(500, 2048, 2)),
    "route of many pairs": lambda: (_route(5000, 64, 4), _route(5000, 2048, 4)),
}


@pytest.mark.parametrize("which", list(PAIRS))
def test_two_threads(which):
    sides = PAIRS[which]()
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    want = []
    for (call, outs), s in zip(sides, streams):
        assert call(s.cuda_stream) == qmoe.QMOE_OK
        s.synchronize()
        want.append([t.clone() for t in outs])
    torch.cuda.synchronize()
    codes = [[], []]
    start = threading.Barrier(2)

    def work(i):
        call, s = sides[i][0], streams[i]
        start.wait()
        for n in range(CALLS):
            codes[i].append(call(s.cuda_stream))
            if n % 50 == 49:
                s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [sorted(set(c)) for c in codes] == [[qmoe.QMOE_OK]] * 2
    for (_, outs), ref in zip(sides, want):
        for t, r in zip(outs, ref):
            assert torch.equal(t, r)
