"""What autograd has to know of the operators' calls: tangents, gradients that a call has none for,
outputs that are written into, and the memory that a call leaves held."""

import gc

import pytest
import torch
import torch.autograd.forward_ad as fw

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe

pytestmark = pytest.mark.gpu

KW = dict(device="cuda", dtype=torch.bfloat16)


def _calls():
    """Of each operator a call of one tensor, and that tensor."""
    t = torch.ones
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(4, 1)
    x, w13, w2, w = t(4, 64, **KW), t(48, 64, **KW), t(64, 24, **KW), t(64, **KW)
    pos = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    weights, rstd = t(4, 2, device="cuda"), t(4, device="cuda")
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, b, scales = t(1, 8, 64, **KW), t(1, 16, 8, **KW), t(1, device="cuda")
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
    return {
        "gate": (lambda v: q.moe_gate(v, 2), x),
        "gate_backward": (lambda v: q.moe_gate_backward(v, x, ids), weights),
        "sort": (lambda v: q.moe_sort_tokens(v, ids, 3), x),
        "sort_backward": (lambda v: q.moe_sort_tokens_backward(v, pos), t(8, 64, **KW)),
        "unsort": (lambda v: q.moe_unsort_tokens(t(8, 64, **KW), pos, v), weights),
        "unsort_backward": (lambda v: q.moe_unsort_tokens_backward(v, t(8, 64, **KW), pos.view(-1), pos,
                                                                   weights), x),
        "lora": (lambda v: q.qmoe_lora_linear(x, None, v, b, one, scales), a),
        "norm": (lambda v: q.qmoe_block_norm(x, post_weight=v), w),
        "norm_backward": (lambda v: q.qmoe_block_norm_backward(v, None, x, post_weight=w,
                                                               post_rstd=rstd), x),
        "checkpoint8": (lambda v: q.qmoe_checkpoint8(v), x),
        "ffn": (lambda v: q.qmoe_gated_ffn(x, v, w2), w13),
        "ffn_saved": (lambda v: q.qmoe_gated_ffn_saved(x, w13, v), w2),
        "ffn_backward": (lambda v: q.qmoe_gated_ffn_backward(v, x, w13, w2, saved), x),
    }


@pytest.mark.parametrize("name", ["gate", "gate_backward", "sort", "sort_backward", "unsort",
                                  "unsort_backward", "lora", "norm", "norm_backward", "checkpoint8",
                                  "ffn", "ffn_saved", "ffn_backward"])
def test_tangents_are_refused(name):
    """None of the operators has a derivative in forward mode: a tangent raises, wherever it is, and
    is not dropped."""
    call, t = _calls()[name]
    call(t)
    with fw.dual_level():
        call(t)  # (no tangent)
        dual = fw.make_dual(t, torch.ones_like(t))
        for guard in (torch.enable_grad(), torch.no_grad()):
            with guard, pytest.raises(NotImplementedError):
                call(dual)
    call(t)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("which", range(3))
def test_the_saved_form_has_no_gradient_and_says_so(which, bits):
    """Its backward pass is its caller's: a gradient that comes to its output raises, as
    qmoe_lora_linear's does, and is not lost."""
    args = [torch.randn(s, **KW) for s in ((5, 64), (48, 64), (64, 24))]
    want, kept = q.qmoe_gated_ffn_saved(*args, checkpoint=bits)
    assert not want.requires_grad
    args[which].requires_grad_(True)
    out, saved = q.qmoe_gated_ffn_saved(*args, checkpoint=bits)
    assert torch.equal(out, want) and out.requires_grad
    assert not any(t.requires_grad for t in saved)
    for a, b in zip(saved, kept):
        assert torch.equal(a, b)
    with pytest.raises(NotImplementedError):
        out.sum().backward()
    with pytest.raises(ValueError):
        q.qmoe_gated_ffn_saved(*args, checkpoint=bits, out=torch.empty_like(want))
    with torch.no_grad():
        out, _ = q.qmoe_gated_ffn_saved(*args, checkpoint=bits, out=torch.empty_like(want))
    assert torch.equal(out, want) and not out.requires_grad


@pytest.mark.parametrize("name", ["norm", "norm_normed", "checkpoint", "restore", "ffn", "lora", "gate",
                                  "sort", "unsort"])
def test_an_output_that_autograd_has_saved(name):
    """A tensor that a node keeps for its backward pass and a call then writes into: the backward pass
    raises, as after any operation in place, in place of a gradient of other values."""
    t = torch.ones
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    pos = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    x, w = t(4, 64, **KW), t(64, **KW)
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    codes, scales = q.qmoe_checkpoint8(x)
    into = {"gate": t(4, 2, device="cuda"), "sort": t(8, 64, **KW), "checkpoint": codes}.get(
        name, t(4, 64, **KW))
    calls = {
        "norm": lambda o: q.qmoe_block_norm(x, residual=o, post_weight=w, out=o),
        "norm_normed": lambda o: q.qmoe_block_norm(x, pre_weight=w, normed=o),
        "checkpoint": lambda o: q.qmoe_checkpoint8(x, codes=o),
        "restore": lambda o: q.qmoe_checkpoint8_restore(codes, scales, out=o),
        "ffn": lambda o: q.qmoe_gated_ffn(x, t(48, 64, **KW), t(64, 24, **KW), out=o),
        "lora": lambda o: q.qmoe_lora_linear(x, None, t(1, 8, 64, **KW), t(1, 64, 8, **KW), one,
                                             t(1, device="cuda"), base=o, out=o),
        "gate": lambda o: q.moe_gate(x, 2, topk_weights=o),
        "sort": lambda o: q.moe_sort_tokens(x, ids, 3, xs=o),
        "unsort": lambda o: q.moe_unsort_tokens(t(8, 64, **KW), pos, t(4, 2, device="cuda"), out=o),
    }
    call = calls[name]
    leaf = torch.ones(into.shape, device="cuda", requires_grad=True)
    product = leaf * into  # keeps `into`
    call(into)
    with pytest.raises(RuntimeError, match="inplace"):
        product.sum().backward()
    # (a refused call has written nothing)
    product, version = leaf * into, into._version
    with pytest.raises((ValueError, qmoe.QmoeError)):
        call(into[1:])
    assert into._version == version
    product.sum().backward()
    with torch.inference_mode():  # tensors without a version
        call(torch.ones_like(into))


def test_an_output_that_requires_a_gradient():
    """What would take the place of its history's values is refused, but under torch.no_grad()."""
    x, w = torch.randn(4, 64, **KW), torch.randn(64, **KW)
    leaf = torch.ones(4, 64, **KW).requires_grad_(True)
    for out in (leaf, leaf * 2):
        with pytest.raises(ValueError):
            q.qmoe_block_norm(x, post_weight=w, out=out)
        with pytest.raises(ValueError):
            q.qmoe_block_norm(x, pre_weight=w, normed=out)
        with torch.no_grad():
            assert torch.equal(q.qmoe_block_norm(x, post_weight=w, out=out)[0],
                               q.qmoe_block_norm(x, post_weight=w)[0])


def _held():
    """Bytes that tensors have asked for.  (memory_allocated counts the allocator's blocks, which it
    splits only where more than 1 MiB would remain.)"""
    gc.collect()
    torch.cuda.synchronize()
    return torch.cuda.memory_stats()["requested_bytes.all.current"]


@pytest.mark.parametrize("bits", [16, 8])
def test_no_workspace_is_held_after_a_call(bits):
    """A gated block's call that brings no workspace leaves its outputs and an error word behind, no
    more (a few allocations of 512 bytes)."""
    M, H, I = 2000, 1024, 512
    x, w13, w2 = (torch.randn(s, **KW) for s in ((M, H), (2 * I, H), (H, I)))

    def step():
        out, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits)
        q.qmoe_gated_ffn_backward(out, x, w13, w2, saved)
        q.qmoe_gated_ffn(x[:3], w13, w2)
        assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)

    _ = q.qmoe_gated_ffn(x[:3], w13, w2)  # the least of workspaces
    tiny = torch.ones(1, 64, **KW)
    small = torch.ones(16, 64, **KW), torch.ones(64, 8, **KW)
    q.qmoe_gated_ffn_backward(tiny, tiny, *small, q.qmoe_gated_ffn_saved(tiny, *small)[1])
    before = _held()
    step()
    assert _held() - before <= 4096
    out, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits)
    before = _held()
    grads = q.qmoe_gated_ffn_backward(out, x, w13, w2, saved)
    held = _held() - before - sum(2 * g.numel() for g in grads)
    assert held <= 4096
