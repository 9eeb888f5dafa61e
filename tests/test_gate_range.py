"""The expert gate where its scores saturate and its choice values are infinite.

Tolerances: u = 2^-24; expf is within 2 ulp (2^-22) for any argument here, a sigmoid and its
complement within 2^-21 then, and the sums of k positive terms add k u.
"""

import math

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q

gpu = pytest.mark.gpu
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("lo,hi", [(8.0, 16.0), (16.0, 30.0), (-30.0, -16.0), (-12.0, 40.0)])
def test_sigmoid_gradient_of_confident_logits(lo, hi, renorm, dtype):
    """s (1 - s) for s next to 1: the complement is not the rounded score's."""
    M, E, k = 64, 48, 6
    g = _gen(int(hi))
    logits = (lo + (hi - lo) * torch.rand(M, E, generator=g, device="cuda")).to(dtype)
    kw = dict(scoring=q.QMOE_GATE_SIGMOID, renormalize=renorm, scale=2.5)
    ids, _ = q.moe_gate(logits, k, **kw)
    dw = torch.randn(M, k, generator=g, device="cuda")
    dl = q.moe_gate_backward(dw, logits, ids, **kw)
    l = torch.gather(logits.double(), 1, ids.long())
    s, rest, d = torch.sigmoid(l), torch.sigmoid(-l), dw.double()
    inner, size, p = 0.0, d.abs(), s
    if renorm:
        p = s / (s.sum(1, keepdim=True) + 1e-20)
        inner = (p * d).sum(1, keepdim=True)
        size = size + (p * d.abs()).sum(1, keepdim=True)
    want = 2.5 * p * rest * (d - inner)
    got = torch.gather(dl, 1, ids.long()).double()
    bound = 2.5 * p * rest * size * (4 * 2.0 ** -21 + (k + 8) * U)
    # what bf16 rounds, and what is below fp32's normal numbers
    bound = bound + torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -126
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / want.abs()).max())
    assert (got[want.abs() > 2.0 ** -120] != 0).all()
    assert torch.count_nonzero(dl) <= M * k


@gpu
@pytest.mark.parametrize("size", [3, 4, 8, 40])  # groups of whole lanes of a warp, and others
def test_group_of_an_infinite_bias_and_masked_experts(size):
    """An infinite choice value beside masked ones: the sum of the two largest is NaN.  The group
    comes first, and no more than topk_group groups are chosen from."""
    G = 4
    l = torch.zeros(3, G * size, device="cuda")
    bias = torch.zeros(G * size, device="cuda")
    bias[2 * size] = math.inf
    l[:, 2 * size + 1:3 * size] = -math.inf
    l[0, size] = 3.0
    l[1, :2 * size] = -math.inf
    l[2, 2 * size] = -math.inf          # the infinite bias masked too
    kw = dict(scoring=q.QMOE_GATE_SIGMOID, bias=bias, n_group=G)
    ids, w = q.moe_gate(l, 2, topk_group=1, **kw)
    assert ids.tolist() == [[2 * size, -1], [2 * size, -1], [0, 1]]
    assert w.tolist() == [[1.0, 0.0], [1.0, 0.0], [0.5, 0.5]]
    ids, _ = q.moe_gate(l, 3, topk_group=2, **kw)
    assert ids.tolist() == [[2 * size, size, size + 1], [2 * size, 3 * size, 3 * size + 1],
                            [0, 1, 2]]


@gpu
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_a_single_renormalized_expert_has_no_gradient(sigmoid, masked):
    """Its weight is `scale` whatever its logit; with masks, rows of top_k 3 with one expert."""
    g = _gen(9)
    M, E, k = 500, 40, 3 if masked else 1
    logits = torch.randn(M, E, generator=g, device="cuda")
    if masked:
        one = torch.randint(0, E, (M, 1), generator=g, device="cuda")
        logits = torch.full_like(logits, -math.inf).scatter_(1, one, logits)
    kw = dict(scoring=int(sigmoid), renormalize=True, scale=2.5)
    ids, w = q.moe_gate(logits, k, **kw)
    assert (w[:, 0] == 2.5).all()
    dl = q.moe_gate_backward(torch.randn(M, k, generator=g, device="cuda"), logits, ids, **kw)
    assert torch.count_nonzero(dl) == 0
