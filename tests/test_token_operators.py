"""The expert gate, the token sort and its inverse, and the projection with adapters:
refusals (CPU) and parity with plain 64-bit forms (GPU).

Tolerances.  u = 2^-24 is fp32's unit roundoff, r the output type's (half its
epsilon: bf16 2^-8, fp16 2^-11 and half a subnormal step of 2^-24, fp32 2^-24).  A sum of n terms in fp32 in any order is within
(n - 1) u sum|terms| of the exact one, plus one rounding per product, so n u sum|terms|
bounds both; tensor-core additions truncate, which doubles u.  expf is within 2 ulp and its
argument l - top within u |l - top|: relative 2^-22 + u |l - top|.  The output's own
rounding adds r |value|.
"""

import ctypes
import math

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

U = 2.0 ** -24
ROUND = {d: torch.finfo(d).eps / 2 for d in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
gpu = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, width, dtype, pad=0, offset=0):
    t = torch.randn(n, width + pad + offset, generator=g, device="cuda").to(dtype)
    return t[:, offset:offset + width]


def _near(got, ref, bound, what):
    got, ref, bound = got.double(), ref.double(), bound.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(),
                           float((got - ref).abs().max()), float(bound[bad].max()))


# ================================================================== refusals, no GPU
@pytest.fixture(scope="module")
def lib():
    from quantized_moe_grouped_route_gb300 import build
    build.build()
    return qmoe.lib()


P = ctypes.c_void_p
ARG, SHAPE, WS, OK = (qmoe.QMOE_ERR_ARG, qmoe.QMOE_ERR_SHAPE, qmoe.QMOE_ERR_WORKSPACE,
                      qmoe.QMOE_OK)


def test_gate_refusals(lib):
    def call(dtype=2, ld=8, M=4, E=8, k=2, scoring=0, bias=None, G=1, tg=1, scale=1.0, ptr=None,
             out=None):
        return lib.moe_gate(ptr, dtype, ld, M, E, k, scoring, bias, G, tg, 1, scale, out, out,
                            None)
    assert call(dtype=3) == ARG and call(dtype=-1) == ARG
    assert call(scoring=2) == ARG
    assert call(scale=math.inf) == ARG and call(scale=math.nan) == ARG
    assert call(E=0) == SHAPE and call(E=2049, ld=2049) == SHAPE
    assert call(k=9) == SHAPE and call(k=0) == SHAPE and call(E=128, ld=128, k=65) == SHAPE
    assert call(ld=7) == SHAPE and call(M=-1) == SHAPE and call(M=1 << 26) == SHAPE
    assert call(G=3) == SHAPE and call(G=0) == SHAPE and call(E=64, ld=64, G=64) == SHAPE
    assert call(G=4, tg=5) == SHAPE and call(G=4, tg=0) == SHAPE
    assert call(G=4, tg=1, k=3) == SHAPE  # more slots than the kept groups hold
    assert call(bias=P(256)) == ARG  # softmax scores take no bias
    assert call() == ARG  # null pointers
    assert call(ptr=P(258), out=P(256)) == ARG  # fp32 logits off a 4-byte boundary
    assert call(M=0) == OK

    def back(dtype=2, ld=8, M=4, E=8, k=2, scoring=0, scale=1.0):
        return lib.moe_gate_backward(None, None, dtype, ld, None, M, E, k, scoring, 1, scale,
                                     None, None)
    assert back(dtype=5) == ARG and back(scoring=-1) == ARG and back(scale=math.inf) == ARG
    assert back(k=9) == SHAPE and back(ld=3) == SHAPE and back() == ARG and back(M=0) == OK


def test_sort_refusals(lib):
    def call(dtype=0, ld=64, M=4, H=64, k=2, E=8, p=None, ws=None, n=1 << 20):
        return lib.moe_sort_tokens(p, dtype, ld, p, M, H, k, E, p, p, p, p, ws, n, None)
    a = P(4096)
    assert call(dtype=9) == ARG and call(H=0) == SHAPE and call(k=65) == SHAPE
    assert call(E=0) == SHAPE and call(E=2049) == SHAPE and call(ld=63) == SHAPE
    assert call(M=1 << 26) == SHAPE and call(M=0) == OK
    assert call(H=(1 << 20) + 1, ld=1 << 21) == SHAPE
    assert call() == ARG and call(p=a, ws=P(4097)) == ARG and call(p=P(4098), ws=a) == ARG
    assert call(p=a, ws=a, n=256) == WS
    assert lib.qmoe_sort_workspace_size(-1, 2, 8) == 0
    assert lib.qmoe_sort_workspace_size(4, 2, 8) >= 256
    assert lib.moe_sort_tokens_backward(None, 0, 64, None, 4, 64, 2, None, None) == ARG
    assert lib.moe_sort_tokens_backward(None, 0, 63, None, 4, 64, 2, None, None) == SHAPE
    assert lib.moe_sort_tokens_backward(None, 0, 64, None, 0, 64, 2, None, None) == OK
    assert lib.moe_unsort_tokens(a, 0, 64, a, None, 4, 64, 2, a, None) == ARG
    assert lib.moe_unsort_tokens(None, 7, 64, None, a, 4, 64, 2, None, None) == ARG
    assert lib.moe_unsort_tokens(None, 0, 64, None, None, 0, 64, 2, None, None) == OK
    back = lib.moe_unsort_tokens_backward
    assert back(None, 64, None, 64, 0, None, None, None, 4, 64, 2, None, None, None) == ARG
    assert back(None, 60, None, 64, 0, None, None, None, 4, 64, 2, None, None, None) == SHAPE
    assert back(None, 64, None, 60, 0, None, None, None, 4, 64, 2, None, None, None) == SHAPE
    assert back(None, 64, None, 64, 0, None, None, None, 0, 64, 2, None, None, None) == OK


def test_lora_refusals(lib):
    a = P(4096)

    def call(dtype=0, ldx=64, M=4, K=64, N=32, R=16, L=4, x=a, w=a, base=None, ldb=0, out=a, ws=a,
             n=1 << 24):
        return lib.qmoe_lora_linear(x, dtype, ldx, w, a, a, a, a, base, ldb, out, M, K, N, R, L,
                                    ws, n, None)
    assert call(dtype=2) == ARG and call(dtype=-1) == ARG
    assert call(K=60) == SHAPE and call(K=0) == SHAPE and call(N=0) == SHAPE
    assert call(R=0) == SHAPE and call(R=12) == SHAPE and call(R=136) == SHAPE
    assert call(L=0) == SHAPE and call(M=-1) == SHAPE
    assert call(ldx=60) == SHAPE and call(ldx=68) == SHAPE and call(base=a, ldb=31) == SHAPE
    assert call(x=None) == ARG and call(x=P(4104)) == ARG and call(w=P(4104)) == ARG
    assert call(ws=P(4100)) == ARG and call(n=16) == WS and call(M=0) == OK
    assert lib.qmoe_lora_workspace_size(4, 60, 32, 16, 4) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.moe_gate(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        q.moe_sort_tokens(x, ids, 8)
    with pytest.raises(ValueError):
        q.qmoe_lora_linear(x, None, x.view(1, 4, 64), x.view(1, 64, 4), ids[:, 0], ids[:, 0])


@gpu
def test_binding_refuses_bad_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        q.moe_gate(x.double(), 2)
    with pytest.raises(ValueError):
        q.moe_gate(x.t(), 2)  # elements of a row apart
    with pytest.raises(ValueError):
        q.moe_gate(x, 2, bias=torch.zeros(8, device="cuda"))
    with pytest.raises(q.QmoeError):
        q.moe_gate(x, 65)
    with pytest.raises(ValueError):
        q.moe_sort_tokens(x, ids.long(), 8)
    with pytest.raises(ValueError):
        q.moe_sort_tokens(x, ids[:3], 8)
    with pytest.raises(q.QmoeError):
        q.moe_sort_tokens(x, ids, 8, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q.moe_unsort_tokens(x, ids, torch.zeros(4, 2, device="cuda"))  # y of 4 rows, not 8
    with pytest.raises(ValueError):
        q.moe_unsort_tokens(x.repeat(2, 1), ids, torch.zeros(4, 2, device="cuda"),
                            out=torch.empty(4, 64, device="cuda"))
    a = torch.zeros(3, 16, 64, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(3, 32, 16, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, device="cuda")
    with pytest.raises(ValueError):
        q.qmoe_lora_linear(x, x, a, b, ids[:, 0].contiguous(), s)  # w of 4 rows, not 32
    with pytest.raises(ValueError):
        q.qmoe_lora_linear(x, None, a.half(), b, ids[:, 0].contiguous(), s)
    with pytest.raises(ValueError):
        q.qmoe_lora_linear(x, None, a, b, ids[:, 0], s)  # ids with a stride


# ============================================================================ gate
def _choice64(logits, sigmoid, bias, G, tg):
    l = logits.double()
    c = torch.sigmoid(l) + (0 if bias is None else bias.double()) if sigmoid else l
    c = torch.where((l > -math.inf) & (c > -math.inf), c, -math.inf)
    if G > 1:
        M, E = l.shape
        v = c.view(M, G, E // G)
        if sigmoid and E // G > 1:
            score = torch.topk(v, 2, dim=-1).values.sum(-1)
        else:
            score = v.amax(-1)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :tg]
        keep = torch.zeros(M, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = torch.where(keep[:, :, None], v, -math.inf).view(M, E)
    return c


def _weights64(logits, ids, sigmoid, renorm, scale):
    """Differentiable in logits (fp64)."""
    there = ids >= 0
    l = torch.gather(logits, 1, ids.clamp(min=0).long())
    if sigmoid:
        s = torch.where(there, torch.sigmoid(l), 0.0)
        w = s / (s.sum(1, keepdim=True) + 1e-20) if renorm else s
    else:
        l = torch.where(there, l, -1e30)
        full = torch.where(logits > -math.inf, logits, -1e30)
        den = torch.logsumexp(l if renorm else full, 1, keepdim=True)
        w = torch.exp(l - den)
    return torch.where(there, w * scale, 0.0)


GATES = [  # M, E, top_k, sigmoid, groups, kept, renormalize
    (1, 1, 1, False, 1, 1, True), (1, 8, 2, False, 1, 1, True), (5, 32, 8, True, 1, 1, True),
    (16, 256, 8, True, 8, 4, True), (33, 60, 4, False, 1, 1, False),
    (7, 129, 6, True, 3, 2, False), (130, 128, 8, False, 4, 2, True),
    (9, 512, 32, True, 32, 9, True), (3, 1024, 33, False, 1, 1, True),
    (2, 2048, 64, True, 16, 16, True), (4, 24, 3, True, 24, 5, True),
    (4, 1000, 64, False, 25, 7, False), (3000, 96, 5, True, 1, 1, True),
]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,E,k,sigmoid,G,tg,renorm", GATES)
def test_gate(M, E, k, sigmoid, G, tg, renorm, dtype):
    g = _gen(M * 7 + E)
    logits = (2 * _rows(g, M, E, torch.float32, pad=3)).to(dtype)
    bias = 0.05 * torch.randn(E, generator=g, device="cuda") if sigmoid else None
    kw = dict(scoring=q.QMOE_GATE_SIGMOID if sigmoid else q.QMOE_GATE_SOFTMAX,
              renormalize=renorm, scale=1.5)
    ids, w = q.moe_gate(logits, k, bias=bias, n_group=G, topk_group=tg, **kw)
    c = _choice64(logits, sigmoid, bias, G, tg)
    want = torch.sort(c, dim=1, descending=True, stable=True)
    if sigmoid:
        # the fp32 choice value is within 8 u of the exact one, a group's score 16 u: equal
        # up to swaps of values nearer than that
        got = torch.gather(c, 1, ids.long())
        same = (ids == want.indices[:, :k]).all(1)
        assert (got[same] - want.values[:, :k][same]).abs().max() == 0
        assert same.double().mean() > 0.99
        near = (got - want.values[:, :k]).abs() <= 32 * U
        assert near[~same].all()
    else:
        assert torch.equal(ids, want.indices[:, :k].to(torch.int32))
    ref = _weights64(logits.double(), ids, sigmoid, renorm, 1.5)
    # exponents up to |l - top| <= 24 and a sum of at most E terms of one sign
    _near(w, ref, ref.abs() * (2.0 ** -21 + (24 + E) * 2 * U), "weights")

    dw = torch.randn(M, k, generator=g, device="cuda")
    dl = q.moe_gate_backward(dw, logits, ids, **kw)
    l64 = logits.double().requires_grad_(True)
    (_weights64(l64, ids, sigmoid, renorm, 1.5) * dw.double()).sum().backward()
    # each term is a product of weights and dw, with cancellation against their sum
    size = 1.5 * (dw.abs().double().amax(1, keepdim=True)) * 2
    bound = size * ((24 + E + k) * 4 * U) + ROUND[dtype] * l64.grad.abs() + TINY[dtype]
    _near(dl, l64.grad, bound.expand_as(l64.grad), "dlogits")


@gpu
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_against_differences(sigmoid, renorm):
    g = _gen(3)
    M, E, k = 6, 40, 5
    logits = torch.randn(M, E, generator=g, device="cuda")
    kw = dict(scoring=int(sigmoid), renormalize=renorm)
    ids, _ = q.moe_gate(logits, k, **kw)
    dw = torch.randn(M, k, generator=g, device="cuda")
    dl = q.moe_gate_backward(dw, logits, ids, **kw).double()
    # a step that keeps the choice: towards the chosen, off the others, second differences
    # of size h^2 and rounding of size u / h
    h = 2.0 ** -8
    d = torch.rand(M, E, generator=g, device="cuda")
    d.scatter_add_(1, ids.long(), torch.ones(M, k, device="cuda"))
    hi, wi = q.moe_gate(logits + h * d, k, **kw)
    lo, wo = q.moe_gate(logits - h * d, k, **kw)
    rows = (hi == ids).all(1) & (lo == ids).all(1)
    assert rows.any()
    num = ((wi.double() - wo.double()) * dw.double()).sum(1) / (2 * h)
    ana = (dl * d.double()).sum(1)
    tol = 8 * dw.abs().double().sum(1) * (h * h + 8 * U / h)
    assert ((num - ana).abs() <= tol)[rows].all(), (num, ana, tol)


@gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate_masks_ties_and_empty_rows(sigmoid):
    inf, nan = math.inf, math.nan
    rows = torch.tensor([
        [0.0, -0.0, 0.0, -0.0, 0.0, 0.0],       # all equal, zeros of both signs
        [1.0, 2.0, 2.0, 1.0, 2.0, 0.0],         # ties at the cut
        [-inf] * 6,                             # nothing left
        [-inf, -inf, 0.5, -inf, -inf, -inf],    # fewer than top_k
        [nan, 1.0, nan, 0.0, -inf, 2.0],        # NaN never chosen
        [-3e38, -3.4e38, -inf, -3.4e38, -inf, -inf],  # the type's lowest values are not masked
        [80.0, -80.0, 100.0, -100.0, 0.0, 3e38],
    ], device="cuda")
    ids, w = q.moe_gate(rows, 3, scoring=int(sigmoid))
    low = [0, 1, 3] if sigmoid else [0, 1, 3]
    top = [[0, 1, 2], [1, 2, 4], [-1, -1, -1], [2, -1, -1], [5, 1, 3], low]
    assert ids.tolist()[:6] == top
    # 100, 80 and 3e38 all have sigmoid 1 in fp32
    assert ids.tolist()[6] == ([0, 2, 5] if sigmoid else [5, 2, 0])
    assert w[2].tolist() == [0.0, 0.0, 0.0] and w[3].tolist() == [1.0, 0.0, 0.0]
    assert torch.isfinite(w).all()
    for r in (0, 1, 4) + (() if sigmoid else (5, 6)):
        assert abs(float(w[r].sum()) - 1.0) < 1e-6
    if sigmoid:  # every score underflows to 0: 0 / 1e-20
        assert w[5].tolist() == [0.0, 0.0, 0.0]
    for renorm in (False, True):
        dl = q.moe_gate_backward(torch.ones(7, 3, device="cuda"), rows, ids,
                                 scoring=int(sigmoid), renormalize=renorm)
        assert torch.isfinite(dl).all()
        assert (dl[2] == 0).all()
        assert (dl[rows == -inf] == 0).all() and (dl[torch.isnan(rows)] == 0).all()
    # every expert at bf16's lowest value is an ordinary tie
    lowest = torch.full((2, 40), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16,
                        device="cuda")
    ids, w = q.moe_gate(lowest, 4, n_group=4, topk_group=2)
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and w.tolist() == [[0.25] * 4] * 2
    # +infinity follows IEEE: NaN weights, valid ids
    ids, w = q.moe_gate(torch.tensor([[0.0, inf, 1.0]], device="cuda"), 2)
    assert ids.tolist() == [[1, 2]]


@gpu
def test_gate_groups_of_masked_experts():
    l = torch.full((3, 12), -math.inf, device="cuda")
    l[0, 5] = 0.0                  # one expert left, in the second of four groups
    l[1, 3:6] = torch.tensor([3.0, -1.0, 0.0], device="cuda")
    l[2, 0] = 9.0                  # a group of one unmasked expert has no second largest
    l[2, 6:9] = 0.0
    ids, w = q.moe_gate(l, 2, scoring=q.QMOE_GATE_SIGMOID, n_group=4, topk_group=1)
    assert ids.tolist() == [[-1, -1], [3, 5], [6, 7]]
    ids, w = q.moe_gate(l, 2, n_group=4, topk_group=1)
    assert ids.tolist() == [[5, -1], [3, 5], [0, -1]]


# ==================================================================== sort, unsort
def _ids(g, M, k, E, dropped=0.0):
    ids = torch.rand(M, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    if dropped:
        ids[torch.rand(M, k, generator=g, device="cuda") < dropped] = -1
    return ids


def _tables(ids, E):
    flat = ids.reshape(-1).tolist()
    order = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    sp = [i for _, i in order] + [-1] * (len(flat) - len(order))
    pp = [-1] * len(flat)
    for pos, (_, i) in enumerate(order):
        pp[i] = pos
    offs = [sum(1 for e, _ in order if e < x) for x in range(E + 1)]
    return offs, sp, pp


TOKENS = [  # M, H, E, top_k, share of pairs dropped, padding, offset of the first element
    (1, 1, 1, 1, 0.0, 0, 0), (1, 8, 4, 2, 0.0, 0, 0), (3, 7, 5, 3, 0.3, 2, 0),
    (16, 7168, 256, 8, 0.0, 0, 0), (17, 1001, 60, 4, 0.2, 0, 0), (65, 264, 8, 8, 0.5, 8, 8),
    (65, 264, 8, 8, 0.0, 8, 1), (40, 2056, 64, 17, 0.1, 0, 0), (2, 4096, 64, 64, 0.0, 0, 0),
    (5, 96, 16, 2, 1.0, 0, 0), (300, 130, 2048, 3, 0.0, 6, 2), (9, 4099, 16, 9, 0.1, 1, 0),
]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,H,E,k,dropped,pad,offset", TOKENS)
def test_sort_and_unsort(M, H, E, k, dropped, pad, offset, dtype):
    g = _gen(M + H)
    ids = _ids(g, M, k, E, dropped)
    x = _rows(g, M, H, dtype, pad, offset)
    xs, offs, sp, pp = q.moe_sort_tokens(x, ids, E)
    o_ref, sp_ref, pp_ref = _tables(ids, E)
    assert offs.tolist() == o_ref and sp.tolist() == sp_ref and pp.reshape(-1).tolist() == pp_ref
    at = sp.clamp(min=0).long() // k
    want = torch.where((sp >= 0)[:, None], x[at], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(xs, want)

    # rows past the routed pairs hold NaN: they are not read
    y = _rows(g, M * k, H, dtype, pad, offset)
    y[int(offs[-1]):] = math.nan
    rows = torch.where((pp >= 0)[..., None], y[pp.clamp(min=0).long()].double(), 0.0)
    dx = q.moe_sort_tokens_backward(y, pp)
    ref, size = rows.sum(1), rows.abs().sum(1)
    _near(dx, ref, k * U * size + ROUND[dtype] * ref.abs() + TINY[dtype], "dx")
    w = torch.rand(M, k, generator=g, device="cuda")
    out = q.moe_unsort_tokens(y, pp, w)
    ref = (rows * w.double()[..., None]).sum(1)
    _near(out, ref, k * U * size + ROUND[dtype] * ref.abs() + TINY[dtype], "out")

    dout = _rows(g, M, H, dtype, pad, offset)
    dy, dw = q.moe_unsort_tokens_backward(dout, y, sp, pp, w)
    pair = sp.clamp(min=0).long()
    ref = torch.where((sp >= 0)[:, None], w.reshape(-1)[pair][:, None] * dout[at].float(), 0.0)
    assert torch.equal(dy, ref.to(dtype))  # one product, one rounding
    prod = rows * dout.double()[:, None, :]
    _near(dw, prod.sum(-1), H * U * prod.abs().sum(-1), "dweights")
    assert (dw[pp < 0] == 0).all()
    # the adjoint: <unsort(y), dout> is linear in y and in w, so it equals <y, dy> and <w, dw>
    # (differences of the operator itself, which the linearity makes exact up to rounding)
    if dtype == torch.float32:
        step = torch.randn(M, k, generator=g, device="cuda")
        diff = (q.moe_unsort_tokens(y, pp, w + step).double()
                - q.moe_unsort_tokens(y, pp, w).double())
        num, ana = (diff * dout.double()).sum(), (dw.double() * step.double()).sum()
        total = (prod.abs().sum(-1) * (w.abs() + step.abs()).double()).sum()
        assert abs(float(num - ana)) <= (H + 4 * k) * 2 * U * float(total) + 1e-30


@gpu
def test_sort_flags_ids_out_of_range():
    x = torch.randn(4, 64, device="cuda")
    ids = torch.tensor([[0, 7], [3, 8], [-1, 2], [2, 1 << 30]], dtype=torch.int32, device="cuda")
    ws = torch.empty(q.qmoe_sort_workspace_size(4, 2, 8), dtype=torch.uint8, device="cuda")
    xs, offs, sp, pp = q.moe_sort_tokens(x, ids, 8, workspace=ws)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_ERR_BAD_ID, qmoe.QMOE_FLAG_BAD_ID)
    assert pp.tolist() == [[0, 4], [3, -1], [-1, 1], [2, -1]] and int(offs[-1]) == 5
    assert (xs[5:] == 0).all()
    q.moe_sort_tokens(x, ids.clamp(max=7), 8, workspace=ws)
    assert qmoe.qmoe_read_error(ws)[0] == qmoe.QMOE_OK
    # positions that no sort of these tokens gives are left out, not followed
    bad = torch.tensor([[0, 1 << 30], [-7, 3], [8, 2], [7, 6]], dtype=torch.int32, device="cuda")
    y = torch.randn(8, 64, device="cuda")
    out = q.moe_unsort_tokens(y, bad, torch.ones(4, 2, device="cuda"))
    assert torch.equal(out, torch.stack([y[0], y[3], y[2], y[7] + y[6]]))


@gpu
def test_sort_matches_route_above_one_block():
    g = _gen(11)
    M, k, E, H = 3001, 8, 256, 24
    ids = _ids(g, M, k, E, 0.05)
    x = _rows(g, M, H, torch.float16)
    xs, offs, sp, pp = q.moe_sort_tokens(x, ids, E)
    o2, s2, p2, _, _, _ = q.moe_route(ids, E, 64)
    assert torch.equal(offs, o2) and torch.equal(sp, s2) and torch.equal(pp.reshape(-1), p2)
    n = int(offs[-1])
    assert torch.equal(xs[:n], x[sp[:n].long() // k]) and (xs[n:] == 0).all()


@gpu
@pytest.mark.parametrize("M,k,E", [(128, 8, 256), (129, 8, 256), (1024, 1, 3), (205, 5, 2048),
                                   (8191, 9, 700), (33000, 4, 2048), (100001, 2, 1)])
def test_sort_tables_match_route(M, k, E):
    """The one-launch sort, one 32-pair step a warp, and several."""
    g = _gen(M)
    ids = torch.randint(-1, E + (E < 2048), (M, k), generator=g, device="cuda",
                        dtype=torch.int32)  # some skipped, some out of range
    x = _rows(g, M, 6, torch.bfloat16)
    ws = torch.empty(q.qmoe_sort_workspace_size(M, k, E), dtype=torch.uint8, device="cuda")
    ws.fill_(0xCD)
    xs, offs, sp, pp = q.moe_sort_tokens(x, ids, E, workspace=ws)
    o2, s2, p2, _, _, ws2 = q.moe_route(ids, E, 64)
    assert torch.equal(offs, o2) and torch.equal(sp, s2) and torch.equal(pp.reshape(-1), p2)
    assert qmoe.qmoe_read_error(ws) == qmoe.qmoe_read_error(ws2)
    n = int(offs[-1])
    assert torch.equal(xs[:n], x[sp[:n].long() // k]) and (xs[n:] == 0).all()


@gpu
@pytest.mark.parametrize("M,E,k", [(257, 256, 8), (64, 2048, 8), (100, 64, 64), (31, 40, 33)])
def test_gate_with_many_equal_logits(M, E, k):
    """Few distinct values: more candidates for the last slots than a warp has lanes."""
    g = _gen(M)
    logits = torch.randint(-1, 2, (M, E), generator=g, device="cuda").float()
    ids, w = q.moe_gate(logits, k)
    assert torch.equal(ids, torch.sort(logits, dim=1, descending=True,
                                       stable=True).indices[:, :k].to(torch.int32))
    logits[torch.rand(M, E, generator=g, device="cuda") < 0.9] = -math.inf
    ids, w = q.moe_gate(logits, k)
    want = torch.sort(logits, dim=1, descending=True, stable=True)
    left = want.values[:, :k] > -math.inf
    assert torch.equal(ids, torch.where(left, want.indices[:, :k], -1).to(torch.int32))
    assert (w[~left] == 0).all()


@gpu
def test_expanded_gradient_and_no_tokens():
    g = _gen(4)
    M, k, E, H = 12, 3, 8, 72
    ids = _ids(g, M, k, E)
    y = _rows(g, M * k, H, torch.bfloat16)
    w = torch.rand(M, k, generator=g, device="cuda")
    _, _, sp, pp = q.moe_sort_tokens(_rows(g, M, H, torch.bfloat16), ids, E)
    one = torch.ones(1, H, dtype=torch.bfloat16, device="cuda")
    a = q.moe_unsort_tokens_backward(one.expand(M, H), y, sp, pp, w)
    b = q.moe_unsort_tokens_backward(one.repeat(M, 1), y, sp, pp, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    none = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    no_ids = torch.empty(0, k, dtype=torch.int32, device="cuda")
    xs, offs, sp, pp = q.moe_sort_tokens(none, no_ids, E)
    assert xs.shape == (0, H) and offs.tolist() == [0] * (E + 1) and pp.shape == (0, k)
    no_w = torch.empty(0, k, device="cuda")
    assert q.moe_unsort_tokens(xs, pp, no_w).shape == (0, H)
    assert q.moe_sort_tokens_backward(xs, pp).shape == (0, H)
    assert q.moe_unsort_tokens_backward(none, xs, sp, pp, no_w)[1].shape == (0, k)
    i, v = q.moe_gate(torch.empty(0, E, device="cuda"), k)
    assert i.shape == (0, k) and v.shape == (0, k)
    assert q.moe_gate_backward(no_w, torch.empty(0, E, device="cuda"), i).shape == (0, E)


@gpu
def test_rows_past_32_bit_offsets():
    M, k, E, H = 40000, 8, 64, 7168  # 2.3e9 elements of pair rows
    g = _gen(8)
    ids = _ids(g, M, k, E)
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    xs, offs, sp, pp = q.moe_sort_tokens(x, ids, E)
    at = torch.tensor([0, M * k // 2, M * k - 2, M * k - 1], device="cuda")
    assert torch.equal(xs[at], x[sp[at].long() // k])
    w = torch.rand(M, k, generator=g, device="cuda")
    out = q.moe_unsort_tokens(xs, pp, w)
    m = torch.tensor([0, 1, M // 2, M - 1], device="cuda")
    ref = x[m].double() * w[m].double().sum(1, keepdim=True)
    size = x[m].double().abs() * w[m].double().sum(1, keepdim=True)
    _near(out[m], ref, k * U * size + ROUND[torch.bfloat16] * ref.abs(), "out")
    del out
    dy, dw = q.moe_unsort_tokens_backward(x, xs, sp, pp, w)
    want = w.reshape(-1)[sp[at].long()][:, None] * x[sp[at].long() // k].float()
    assert torch.equal(dy[at], want.to(torch.bfloat16))
    sq = x[m].double().square().sum(1, keepdim=True).expand(4, k)
    _near(dw[m], sq, H * U * sq, "dweights")


# ======================================================================== adapters
LORAS = [  # M, K, N, R, L, with w, with base, ids
    (1, 8, 1, 8, 1, True, False, "mixed"), (1, 7168, 2048, 16, 32, True, False, "mixed"),
    (3, 72, 130, 24, 5, True, True, "mixed"), (16, 512, 257, 8, 3, False, True, "mixed"),
    (17, 1000, 99, 128, 4, True, False, "mixed"), (64, 264, 512, 40, 64, True, True, "mixed"),
    (129, 520, 384, 64, 7, True, False, "runs"), (300, 1032, 515, 16, 9, True, True, "runs"),
    (257, 64, 128, 16, 300, True, False, "mixed"), (40, 4096, 64, 32, 2, False, False, "runs"),
    (70, 136, 200, 16, 4, True, False, "none"), (513, 2048, 1000, 32, 6, True, False, "mixed"),
]


# enough tokens times ranks that x . A^T runs on the tensor cores: adapters stacked 1 to 16
# at a time, more of them than one pass holds, a rank that does not divide the 128 rows
LORAS_WIDE = [
    (256, 4096, 96, 24, 40, True, False, "mixed"), (200, 2048, 130, 128, 50, True, False, "mixed"),
    (1100, 1024, 300, 8, 500, True, True, "mixed"), (33, 8192, 64, 64, 9, False, True, "mixed"),
    (2047, 1096, 512, 48, 11, True, False, "runs"), (60, 256, 20000, 64, 40, True, True, "mixed"),
    (31, 512, 160, 128, 31, True, False, "mixed"), (2, 2056, 77, 128, 2, True, True, "mixed"),
    (4, 4104, 130, 72, 9, True, False, "mixed"), (3, 1544, 5, 32, 2, False, False, "mixed"),
    (1, 16384, 40, 64, 3, True, True, "runs"), (8, 4104, 77, 128, 9, True, True, "mixed"),
    (7, 40, 17, 8, 3, True, False, "mixed"), (5, 16400, 31, 24, 2, True, False, "runs"),
    (8, 8200, 4099, 64, 30, True, False, "mixed"), (6, 2048, 100, 40, 5, False, True, "mixed"),
    (2, 8192, 48, 128, 2, True, False, "none"), (64, 1024, 30000, 16, 60, True, False, "mixed"), (700, 968, 200, 128, 3, True, False, "none"),
]


# many adapters a tile, in every length of the tensor-core operand's rows, over several tiles a
# CTA; ranks that end inside a step of 64, or inside the 16 of an MMA
LORAS_MANY = [
    (128, 256, 1100, 16, 90, True, False, "mixed"), (120, 72, 300, 8, 40, True, True, "mixed"),
    (480, 136, 20000, 72, 30, True, False, "mixed"), (600, 128, 12000, 24, 60, True, False, "mixed"),
    (400, 128, 16000, 8, 20, True, False, "runs"), (250, 64, 700, 32, 200, False, True, "mixed"),
    (1000, 64, 9000, 40, 12, True, False, "mixed"), (48, 128, 500, 104, 30, True, False, "mixed"),
    (256, 200, 12000, 24, 40, True, True, "mixed"), (1020, 520, 4096, 64, 30, True, False, "mixed"),
    (250, 16, 70, 8, 5000, True, False, "mixed"),
    # few token-ranks, adapters enough for one a token (and not): fp32 products beside w
    (48, 1024, 300, 32, 64, True, False, "mixed"), (30, 520, 260, 40, 33, True, True, "mixed"),
    (16, 264, 130, 96, 20, False, True, "mixed"), (64, 264, 512, 24, 64, True, True, "mixed"),
    (64, 136, 384, 8, 5, True, False, "mixed"), (40, 264, 20000, 32, 50, True, False, "mixed"),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N,R,L,with_w,with_base,how", LORAS + LORAS_WIDE + LORAS_MANY)
def test_lora_linear(M, K, N, R, L, with_w, with_base, how, dtype):
    g = _gen(M * 3 + K)
    x = _rows(g, M, K, dtype, pad=8)
    w = (_rows(g, N, K, torch.float32) * K ** -0.5).to(dtype) if with_w else None
    a = (_rows(g, L * R, K, torch.float32) * K ** -0.5).to(dtype).view(L, R, K)
    b = (_rows(g, L * N, R, torch.float32) * R ** -0.5).to(dtype).view(L, N, R)
    s = 0.5 + torch.rand(L, generator=g, device="cuda")
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    if how == "runs":
        ids = ids.sort().values.contiguous()
    elif how == "none":
        ids.fill_(-1)
    base = _rows(g, M, N, dtype, pad=5) if with_base else None
    # adapters that no token uses hold NaN: they are not read into a result
    unused = torch.ones(L, dtype=torch.bool, device="cuda")
    unused[ids[ids >= 0].long()] = False
    a[unused], b[unused], s[unused] = math.nan, math.nan, math.nan
    ws = torch.empty(q.qmoe_lora_workspace_size(M, K, N, R, L), dtype=torch.uint8, device="cuda")
    ws.fill_(0xAB)
    out = q.qmoe_lora_linear(x, w, a, b, ids, s, base=base, workspace=ws)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
    ref = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    x64 = x.double()
    if with_base:
        ref += base.double()
        size += base.double().abs()
    if with_w:
        ref += x64 @ w.double().t()
        size += x64.abs() @ w.double().abs().t()
    low = torch.zeros_like(ref)  # bound of the rounding of t, relative to |t|
    for i in range(L):
        m = (ids == i).nonzero()[:, 0]
        if m.numel():
            ai, bi, si = a[i].double(), b[i].double(), s[i].double()
            t = si * (x64[m] @ ai.t())
            ref[m] += t @ bi.t()
            size[m] += si * ((x64[m].abs() @ ai.abs().t()) @ bi.abs().t())
            low[m] += t.abs() @ bi.abs().t()
    # truncating tensor-core sums of K + R terms; t kept to 16 significant bits or more
    bound = (K + R + 4) * 2 * U * size + 2.0 ** -16 * low + ROUND[dtype] * ref.abs() + TINY[dtype]
    _near(out, ref, bound, "out")
    again = q.qmoe_lora_linear(x, w, a, b, ids, s, base=base)
    assert torch.equal(out, again)
    if with_base:  # the result in place of the base
        inout = base.contiguous()
        q.qmoe_lora_linear(x, w, a, b, ids, s, base=inout, out=inout)
        assert torch.equal(inout, out)


@gpu
@pytest.mark.parametrize("M,R", [(20, 16), (100, 16), (128, 32), (70, 64), (300, 24), (260, 120)])
def test_lora_token_of_infinities_stays_alone(M, R):
    """A token whose x A^T is infinite or NaN spoils its own row and no other."""
    K, N, L = 128, 1500, 12
    g = _gen(M + R)
    x = _rows(g, M, K, torch.bfloat16)
    w = _rows(g, N, K, torch.bfloat16)
    a, b = _rows(g, L * R, K, torch.bfloat16), _rows(g, L * N, R, torch.bfloat16)
    s = torch.ones(L, device="cuda")
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    args = (w, a.view(L, R, K), b.view(L, N, R), ids, s)
    good = q.qmoe_lora_linear(x, *args)
    at = torch.arange(3, M, 7, device="cuda")
    x[at[::2], 5], x[at[1::2], 5] = math.inf, math.nan
    out = q.qmoe_lora_linear(x, *args)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(out[keep], good[keep])
    assert not torch.isfinite(out[at]).any()


@gpu
def test_lora_flags_ids_out_of_range():
    g = _gen(2)
    M, K, N, R, L = 20, 128, 96, 16, 3
    x, w = _rows(g, M, K, torch.bfloat16), _rows(g, N, K, torch.bfloat16)
    a = _rows(g, L * R, K, torch.bfloat16).view(L, R, K)
    b = _rows(g, L * N, R, torch.bfloat16).view(L, N, R)
    s = torch.ones(L, device="cuda")
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    bad = ids.clone()
    bad[3], bad[11], bad[12] = L, 1 << 30, -(1 << 30)
    none = ids.clone()
    none[[3, 11, 12]] = -1
    ws = torch.empty(q.qmoe_lora_workspace_size(M, K, N, R, L), dtype=torch.uint8, device="cuda")
    got = q.qmoe_lora_linear(x, w, a, b, bad, s, workspace=ws)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_ERR_BAD_ID, qmoe.QMOE_FLAG_BAD_ID)
    assert torch.equal(got, q.qmoe_lora_linear(x, w, a, b, none, s, workspace=ws))
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
    empty = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    assert q.qmoe_lora_linear(empty, w, a, b, ids[:0], s).shape == (0, N)


# ================================================================ streams and graphs
@gpu
def test_on_another_stream_and_in_a_graph():
    g = _gen(6)
    M, E, k, H, N, R, L = 48, 64, 6, 512, 384, 16, 8
    logits = torch.randn(M, E, generator=g, device="cuda")
    x = _rows(g, M, H, torch.bfloat16)
    w = (_rows(g, N, H, torch.float32) * H ** -0.5).bfloat16()
    a = (_rows(g, L * R, H, torch.float32) * H ** -0.5).bfloat16().view(L, R, H)
    b = _rows(g, L * N, R, torch.bfloat16).view(L, N, R)
    s = torch.ones(L, device="cuda")
    ad = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)

    def chain(stream=None):
        ids, wts = q.moe_gate(logits, k, stream=stream)
        xs, _, sp, pp = q.moe_sort_tokens(x, ids, E, stream=stream)
        out = q.moe_unsort_tokens(xs, pp, wts, stream=stream)
        dy, dw = q.moe_unsort_tokens_backward(out, xs, sp, pp, wts, stream=stream)
        dx = q.moe_sort_tokens_backward(dy, pp, stream=stream)
        dl = q.moe_gate_backward(dw, logits, ids, stream=stream)
        y = q.qmoe_lora_linear(dx, w, a, b, ad, s, stream=stream)
        return [ids, wts, xs, out, dy, dw, dx, dl, y]

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        got = chain(given)
        side.synchronize()
        for u, v in zip(want, got):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    logits.neg_()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(chain(), got):
        assert torch.equal(u, v)
