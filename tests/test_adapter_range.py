"""The projection with adapters over the range of its definition: t = scales[a] (x A[a]^T) far
from 1, and what a request gets next to other requests.

Tolerances as in test_token_operators.py.  Beyond eight tokens t enters the MMA with an error
of at most 2^-16 of the largest of the eight ranks that share a 16-byte unit (bf16: of each
value; fp16: half a subnormal step, 2^-25, where that largest is at least 2^-9).
"""

import math

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

U = 2.0 ** -24
ROUND = {d: torch.finfo(d).eps / 2 for d in (torch.bfloat16, torch.float16)}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
gpu = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _exact(x, w, a, b, ids, s, base=None):
    """(out, the sizes of its sums' terms, the bound of t's rounding) in 64 bits."""
    M, N, R = x.shape[0], b.shape[1], b.shape[2]
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    size, low = torch.zeros_like(out), torch.zeros_like(out)
    x = x.double()
    if base is not None:
        out += base.double()
        size += base.double().abs()
    if w is not None:
        out += x @ w.double().t()
        size += x.abs() @ w.double().abs().t()
    for i in range(a.shape[0]):
        m = (ids == i).nonzero()[:, 0]
        if m.numel():
            ai, bi, si = a[i].double(), b[i].double(), s[i].double()
            t = si * (x[m] @ ai.t())
            out[m] += t @ bi.t()
            size[m] += si * ((x[m].abs() @ ai.abs().t()) @ bi.abs().t())
            top = t.abs().view(-1, R // 8, 8).amax(2, keepdim=True).expand(-1, -1, 8)
            low[m] += top.reshape(-1, R) @ bi.abs().t()
    return out, size, low


def _near(got, x, w, a, b, ids, s, base=None):
    ref, size, low = _exact(x, w, a, b, ids, s, base)
    K, R, dt = x.shape[1], b.shape[2], x.dtype
    bound = ((K + R + 4) * 2 * U * size + 2.0 ** -16 * low + ROUND[dt] * ref.abs() + TINY[dt])
    assert ref.abs().max() < torch.finfo(dt).max
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((got.double() - ref).abs().max()))


RANGES = [  # M, K, N, R, L, with w, with base: every form of the projection above eight tokens
    (20, 256, 260, 16, 3, True, False), (100, 512, 130, 16, 5, True, True),
    (128, 1024, 384, 64, 90, False, False), (70, 136, 200, 24, 4, False, True),
    (300, 264, 515, 8, 9, True, False), (1100, 128, 300, 40, 6, False, False),
    (256, 4096, 96, 24, 40, True, False), (600, 2048, 640, 128, 3, True, True),
    # fp32 products beside w, at the edges of their range
    (16, 256, 260, 64, 16, True, False), (32, 264, 260, 32, 40, True, True),
    (64, 1024, 300, 16, 64, False, False), (64, 264, 512, 8, 5, True, False),
    (32, 264, 260, 40, 40, True, False), (16, 136, 130, 72, 20, True, True),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size_t", [1e5, 3e4, 1e-3, 1e-5, 1e-7])
@pytest.mark.parametrize("M,K,N,R,L,with_w,with_base", RANGES)
def test_t_far_from_one(M, K, N, R, L, with_w, with_base, size_t, dtype):
    """Half the adapters have t of the given size (and B so that the result is of size 1 or
    2^-10 and more), the others of size 1."""
    g = _gen(M + K)
    x = _randn(g, M, K).to(dtype)
    w = _randn(g, N, K, std=K ** -0.5).to(dtype) if with_w else None
    a = _randn(g, L * R, K, std=K ** -0.5).to(dtype).view(L, R, K)
    big = min(max(1.0 / size_t, 1e-4), 4096.0)  # fp16 holds it
    far = (torch.arange(L, device="cuda") % 2 == 0)[:, None, None]
    b = (_randn(g, L, N, R, std=R ** -0.5) * torch.where(far, big, 1.0)).to(dtype)
    s = torch.where(far[:, 0, 0], size_t, 1.0).float() * (0.5 + torch.rand(L, generator=g,
                                                                           device="cuda"))
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    base = _randn(g, M, N).to(dtype) if with_base else None
    out = q.qmoe_lora_linear(x, w, a, b, ids, s, base=base)
    assert torch.isfinite(out).all()
    _near(out, x, w, a, b, ids, s, base)
    again = q.qmoe_lora_linear(x, w, a, b, ids, s, base=base)
    assert torch.equal(out, again)
    # the same requests in batches of eight and one: the same result, each within its bound
    for lo, n in ((0, 8), (8, 1), (M - 8, 8)):
        part = slice(lo, lo + n)
        few = q.qmoe_lora_linear(x[part], w, a, b, ids[part].contiguous(), s,
                                 base=None if base is None else base[part])
        _near(few, x[part], w, a, b, ids[part], s, None if base is None else base[part])


@gpu
@pytest.mark.parametrize("M,R", [(100, 16), (128, 64), (300, 24), (260, 120)])
def test_t_of_all_sizes_in_one_token(M, R):
    """Ranks of one token from 2^-30 to 2^20: those that share a unit, and neighbours."""
    g = _gen(R)
    K, N, L, dtype = 64, 200, 3, torch.float16
    x = _randn(g, M, K).to(dtype)
    x[3] = 0  # t of zero takes no part
    e = torch.randint(-14, 3, (L, R, 1), generator=g, device="cuda").float()
    e[1, 8:] = -14.0  # whole units of small values
    a = (_randn(g, L, R, K, std=K ** -0.5) * 2.0 ** e).to(dtype)
    s = torch.tensor([2.0 ** 17, 2.0 ** -16, 1.0], device="cuda")
    b = _randn(g, L, N, R).to(dtype)
    b[0] = (b[0].float() * 2.0 ** -14).to(dtype)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    for w in (None, _randn(g, N, K, std=K ** -0.5).to(dtype)):
        out = q.qmoe_lora_linear(x, w, a, b, ids, s)
        _near(out, x, w, a, b, ids, s)


SPOILED = [  # M, K, N, R, L, with w, with base: few tokens, one tile with K split and not, pairs
    (1, 256, 130, 16, 2, True, False), (7, 512, 130, 16, 3, True, True),
    (30, 520, 260, 40, 33, True, True), (20, 256, 300, 128, 6, True, False),
    (100, 64, 200, 24, 6, True, True), (128, 1024, 384, 16, 40, True, False),
    (70, 136, 203, 64, 4, False, True), (128, 200, 20000, 16, 60, True, False),
    (200, 264, 515, 8, 9, True, True), (300, 4096, 256, 32, 5, True, False),
    (1100, 136, 4099, 40, 30, True, False), (2047, 1096, 4096, 16, 8, True, True),
    (513, 64, 70, 72, 300, False, False),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N,R,L,with_w,with_base", SPOILED)
def test_adapter_of_infinities_stays_alone(M, K, N, R, L, with_w, with_base, dtype):
    """Infinities and NaN in one adapter's B reach its own tokens, in their columns, and no
    other token."""
    g = _gen(M + N)
    x = _randn(g, M, K).to(dtype)
    w = _randn(g, N, K, std=K ** -0.5).to(dtype) if with_w else None
    a = _randn(g, L * R, K, std=K ** -0.5).to(dtype).view(L, R, K)
    b = _randn(g, L, N, R, std=R ** -0.5).to(dtype)
    s = 0.5 + torch.rand(L, generator=g, device="cuda")
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[M // 2] = L - 1
    base = _randn(g, M, N).to(dtype) if with_base else None
    good = q.qmoe_lora_linear(x, w, a, b, ids, s, base=base)
    bad = b.clone()
    rows = torch.tensor(sorted({0, 3, 33, 64, N // 2, N - 2, N - 1}), device="cuda")
    values = torch.tensor([math.inf, math.nan, -math.inf], device="cuda")
    for i, n in enumerate(rows.tolist()):
        bad[L - 1, n, (5 * i) % R] = values[i % 3]
    ws = torch.empty(q.qmoe_lora_workspace_size(M, K, N, R, L), dtype=torch.uint8, device="cuda")
    out = q.qmoe_lora_linear(x, w, a, bad, ids, s, base=base, workspace=ws)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
    others = ids != L - 1
    assert others.any() or M == 1
    assert torch.isfinite(out[others]).all()
    if others.any():
        _near(out[others], x[others], w, a, b, ids[others], s,
              None if base is None else base[others])
    clean = torch.ones(N, dtype=torch.bool, device="cuda")
    clean[rows] = False
    assert torch.equal(out[:, clean], good[:, clean])
    # its own tokens: an infinity times t, with t's sign
    mine = (~others).nonzero()[:, 0]
    t = x[mine].double() @ a[L - 1].double().t()
    for i, n in enumerate(rows.tolist()):
        ti = t[:, (5 * i) % R]
        sure = ti.abs() > 1e-3
        got, v = out[mine, n], float(values[i % 3])
        if math.isnan(v):
            assert torch.isnan(got).all()
        else:
            assert torch.equal(got[sure].double(), torch.sign(ti[sure]) * v)
    again = q.qmoe_lora_linear(x, w, a, bad, ids, s, base=base)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(again))
    if with_base:  # in place of the base
        inout = base.clone()
        q.qmoe_lora_linear(x, w, a, bad, ids, s, base=inout, out=inout)
        assert torch.equal(torch.nan_to_num(inout), torch.nan_to_num(out))


@gpu
@pytest.mark.parametrize("M", [100, 300])
def test_infinities_everywhere(M):
    """A token of NaN, a row of w of infinities and an adapter of NaN, each in its place."""
    g = _gen(M)
    K, N, R, L, dtype = 128, 520, 16, 4, torch.bfloat16
    x, w = _randn(g, M, K).to(dtype), _randn(g, N, K, std=K ** -0.5).to(dtype)
    a = _randn(g, L * R, K, std=K ** -0.5).to(dtype).view(L, R, K)
    b = _randn(g, L, N, R).to(dtype)
    s = torch.ones(L, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % L
    want = q.qmoe_lora_linear(x, w, a, b, ids, s)
    x[0, 7], w[5], b[2] = math.nan, math.inf, math.nan
    a[3] = math.nan
    out = q.qmoe_lora_linear(x, w, a, b, ids, s)
    there = (ids < 2)[:, None].expand(M, N).clone()
    there[0], there[:, 5] = False, False
    # rows of w beside b's NaN are added up anew, so equal up to rounding
    assert torch.isfinite(out[there]).all() and not torch.isfinite(out[~there]).any()
    err = (out.double() - want.double()).abs()[there]
    assert (err <= 2.0 ** -7 * want.double().abs()[there] + 2.0 ** -10).all()


@pytest.mark.parametrize("K,N,R", [(4096, 4096, 16), (7168, 2048, 64), (2048, 7168, 32), (64, 64, 8),
                                   (1096, 512, 128), (65536, 131072, 128)])
def test_workspace_serves_every_smaller_batch(K, N, R):
    from quantized_moe_grouped_route_gb300 import build
    build.build()
    sizes = [q.qmoe_lora_workspace_size(M, K, N, R, 8) for M in range(1, 9000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    # and of fewer ranks or a shorter K; what it holds is in proportion to the batch
    for M in (1, 100, 513, 5152, 8192):
        assert q.qmoe_lora_workspace_size(M, K // 2 // 8 * 8, N, R, 8) <= sizes[M - 1]
        assert R == 8 or q.qmoe_lora_workspace_size(M, K, N, R - 8, 8) <= sizes[M - 1]
        assert sizes[M - 1] <= 4 * (9 * M * R + 4 * (M + 256)) + 16 * 256
