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


def _block(logits, x, experts, top_k, unsort, sort, gate):
    """A mixture of one-matrix experts through the three operators."""
    E = experts.shape[0]
    ids, weights = gate(logits, top_k)
    xs, offsets, _, pair_pos = sort(x, ids, E)
    ends = offsets.tolist()
    y = torch.cat([xs[ends[e]:ends[e + 1]] @ experts[e].t() for e in range(E)]
                  + [xs[ends[E]:]])
    return unsort(y, pair_pos, weights), ids


@gpu
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_reach_torch(masked):
    """loss.backward() through the operators against autograd of the definition in 64 bits.
    fp32 sums of at most H = 24 and top_k terms: a relative error of 2^-16 of the largest is
    far above their rounding."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, E, H, k = 40, 6, 24, 3
    logits = torch.randn(M, E, generator=g, device="cuda")
    if masked:
        logits[torch.rand(M, E, generator=g, device="cuda") < 0.5] = -torch.inf
        logits[3] = -torch.inf
    x = torch.randn(M, H, generator=g, device="cuda")
    experts = torch.randn(E, H, H, generator=g, device="cuda")
    c = torch.randn(M, H, generator=g, device="cuda")
    mine = [t.clone().requires_grad_(True) for t in (logits, x, experts)]
    out, ids = _block(*mine, k, q.moe_unsort_tokens, q.moe_sort_tokens, q.moe_gate)
    (out * c).sum().backward()
    l64, x64, e64 = (t.double().requires_grad_(True) for t in (logits, x, experts))
    there = (ids >= 0)
    at = ids.clamp(min=0).long()
    l = torch.where(there, torch.gather(l64, 1, at), -1e30)
    w = torch.where(there, torch.softmax(l, 1), 0.0)
    ref = (w[..., None] * torch.einsum("mh,mkoh->mko", x64, e64[at])).sum(1)
    (ref * c.double()).sum().backward()
    for got, want in zip((out, *[t.grad for t in mine]), (ref, l64.grad, x64.grad, e64.grad)):
        want = torch.nan_to_num(want.detach())
        assert got.shape == want.shape
        assert (got.double() - want).abs().max() <= 2.0 ** -16 * want.abs().max()


@gpu
def test_gradients_are_the_explicit_calls():
    g = torch.Generator(device="cuda").manual_seed(6)
    M, E, H, k = 33, 16, 40, 4
    logits = torch.randn(M, E, generator=g, device="cuda").bfloat16().requires_grad_(True)
    bias = torch.randn(E, generator=g, device="cuda").requires_grad_(True)
    kw = dict(scoring=q.QMOE_GATE_SIGMOID, scale=2.5)
    ids, w = q.moe_gate(logits, k, bias=bias, n_group=4, topk_group=2, **kw)
    dw = torch.randn(M, k, generator=g, device="cuda")
    w.backward(dw)
    assert bias.grad is None and not ids.requires_grad
    with torch.no_grad():
        assert torch.equal(logits.grad, q.moe_gate_backward(dw, logits, ids, **kw))
        ids[::3, 1] = -1
    x = torch.randn(M, H, generator=g, device="cuda").half().requires_grad_(True)
    xs, _, sp, pp = q.moe_sort_tokens(x, ids, E)
    xs.sum().backward()  # an expanded gradient
    assert torch.equal(x.grad, q.moe_sort_tokens_backward(torch.ones_like(xs), pp))
    y = torch.randn(M * k, H, generator=g, device="cuda").half().requires_grad_(True)
    w = w.detach().requires_grad_(True)
    dout = torch.randn(H, M, generator=g, device="cuda").half()
    q.moe_unsort_tokens(y, pp, w).backward(dout.t())
    dy, dw = q.moe_unsort_tokens_backward(dout.t().contiguous(), y.detach(), sp, pp, w.detach())
    assert torch.equal(y.grad, dy) and torch.equal(w.grad, dw)


@gpu
def test_what_autograd_cannot_have_is_refused():
    t = torch.ones
    kw = dict(device="cuda", dtype=torch.bfloat16)
    s, ids = torch.ones(2, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    base = t(4, 16, **kw)
    args = [t(4, 64, **kw), t(16, 64, **kw), t(2, 8, 64, **kw), t(2, 16, 8, **kw)]
    want = q.qmoe_lora_linear(*args, ids, s, base=base)
    for i in range(4):
        some = list(args)
        some[i] = some[i].clone().requires_grad_(True)
        out = q.qmoe_lora_linear(*some, ids, s, base=base)
        assert torch.equal(out, want) and out.requires_grad
        with pytest.raises(NotImplementedError):
            out.sum().backward()
        with pytest.raises(ValueError):
            q.qmoe_lora_linear(*some, ids, s, base=base, out=torch.empty_like(base))
        with torch.no_grad():
            out = q.qmoe_lora_linear(*some, ids, s, base=base, out=torch.empty_like(base))
        assert torch.equal(out, want) and not out.requires_grad
    assert not want.requires_grad
    with pytest.raises(ValueError):
        q.moe_gate(t(4, 8, device="cuda", requires_grad=True), 2,
                   topk_weights=t(4, 2, device="cuda"))
    x = t(4, 8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):  # a call's own refusals stay
        q.moe_gate(x.t()[:, ::2], 2)


@gpu
def test_a_flag_without_a_truth_value():
    logits = torch.zeros(4, 8, device="cuda")
    both = torch.tensor([True, False])
    with pytest.raises(RuntimeError, match="ambiguous"):
        q.moe_gate(logits, 2, renormalize=both)
    ids, w = q.moe_gate(logits, 2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        q.moe_gate_backward(w, logits, ids, renormalize=both)
