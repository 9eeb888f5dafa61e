"""What autograd has to know of the operators' calls: tangents, gradients that a call has none for,
outputs that are written into, and the memory that a call leaves held."""

import pytest
import torch
import torch.autograd.forward_ad as fw

import quantized_moe_grouped_route_gb300 as q

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
