"""The dense side of a block (binding of the same-named C-ABI calls): the norms around it fused with
its gate and residual, the gated feed-forward block (a shared expert next to the layer's, or a
dense layer's), and activation checkpoints in 8 bits.

Tensors, streams, workspaces and errors as in operators.py.  Activations' rows may lie apart (the
gated feed-forward block wants each 16-byte aligned and its own); weights are contiguous.

Autograd: qmoe_block_norm and qmoe_gated_ffn on tensors that require a gradient are nodes of its
graph, whose backward is the *_backward call of the same name (those calls and the checkpoints have
no derivative of their own).  qmoe_gated_ffn_saved leaves the backward pass to its caller: a gradient
that comes to its output raises NotImplementedError.  Such a call takes no outputs to write into.
A backward pass that is captured into a CUDA graph must find no eager graph of the same leaves
alive: PyTorch would have it wait for the eager one's stream, which a capture cannot.
"""

from __future__ import annotations

import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import operators, qmoe
from .operators import _native, _on, _rows

QMOE_GATING_LINEAR = 0
QMOE_GATING_SIGMOID = 1
QMOE_ACT_SILU = 0
QMOE_ACT_GELU = 1


# ------------------------------------------------------------------------ autograd
class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, gate, gating, post_weight, pre_weight, residual_scale,
                weight_offset, eps, *outputs):
        out, normed, post_rstd, pre_rstd = _native().block_norm(
            y, residual, gate, gating, post_weight, pre_weight, residual_scale, weight_offset, eps,
            *outputs)
        ctx.save_for_backward(y, out, gate, post_weight, pre_weight, post_rstd, pre_rstd)
        ctx.how = (gating, residual_scale, weight_offset)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*(t for t in (post_rstd, pre_rstd) if t is not None))
        return out, normed, post_rstd, pre_rstd

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dnormed, *_):
        if dout is None and dnormed is None:
            return 11 * (None,)
        y, out, gate, post_weight, pre_weight, post_rstd, pre_rstd = ctx.saved_tensors
        gating, residual_scale, weight_offset = ctx.how
        if dnormed is None:  # of the norm nothing was used
            pre_weight, pre_rstd = None, None
        need = ctx.needs_input_grad
        grads = _native().block_norm_backward(
            None if dout is None else _rows(dout), None if dnormed is None else _rows(dnormed), y,
            out, gate, gating, post_weight, pre_weight, residual_scale, weight_offset, post_rstd,
            pre_rstd, need[1], need[2], need[4], need[5], True)
        dy, dresidual, dgate, dpost, dpre = grads
        return dy, dresidual, dgate, None, dpost, dpre, None, None, None, None, None


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2, activation, limit, _, out, workspace, checkpoint):
        out, *kept = _native().gated_ffn(x, w13, w2, activation, limit, checkpoint, out, workspace, 0)
        held = _native().checkpoint8(x, None, None) if checkpoint == 8 else (x, None)
        ctx.save_for_backward(w13, w2, *kept, *held)
        ctx.how = (activation, limit)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        w13, w2, kept, kept_scales, x, x_scales = ctx.saved_tensors
        dx, dw13, dw2 = _native().gated_ffn_backward(
            _aligned(dout), x, x_scales, w13, w2, kept, kept_scales, *ctx.how,
            *ctx.needs_input_grad[:3], None)
        return (dx, dw13, dw2) + 6 * (None,)


class _GatedFfnSaved(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *args):
        out, *kept = _native().gated_ffn(*args)
        ctx.mark_non_differentiable(*(t for t in kept if t is not None))
        return (out, *kept)

    @staticmethod
    def backward(ctx, *_):
        raise NotImplementedError("qmoe_gated_ffn_saved leaves the backward pass to its caller: call it "
                                  "under torch.no_grad() or on detached tensors, or qmoe_gated_ffn")


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the gated block takes rows: 16-byte aligned, and each its own."""
    t = _rows(t)
    apart = t.stride(0) if t.size(0) > 1 else t.size(1)
    fits = apart >= t.size(1) and apart % 8 == 0 and t.data_ptr() % 16 == 0
    return t if fits else t.clone(memory_format=torch.contiguous_format)


# of each call the node, and which of its arguments are outputs
operators._NODES.update({"block_norm": (_BlockNorm, (9, 10)), "gated_ffn": (_GatedFfn, (6,)),
                         "gated_ffn_saved": (_GatedFfnSaved, (6,))})


# --------------------------------------------------------------- norms around a block
def qmoe_block_norm(y: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
                    gate: Optional[torch.Tensor] = None, gating: int = QMOE_GATING_LINEAR,
                    post_weight: Optional[torch.Tensor] = None,
                    pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                    weight_offset: float = 0.0, eps: float = 1e-6,
                    out: Optional[torch.Tensor] = None, normed: Optional[torch.Tensor] = None,
                    stream=None):
    """The norm after a block, its gate, the residual and the norm before the next block:
    out = residual_scale residual + gate rms(y) (weight_offset + post_weight), normed =
    rms(out) (weight_offset + pre_weight), rms(v) = v / sqrt(mean(v^2) + eps).

    y, residual [M][H]; gate [M][1], [1][H] or [M][H] of their dtype or fp32 (gating: as given, or
    its sigmoid; [1][H] is a channel's also of one token); weights [H] of their dtype or fp32; any of them may
    be None, without which the part is left out.  Returns (out, normed, post_rstd, pre_rstd), the
    last two fp32 [M] for the backward pass; None for what there is not (out: where it would be y).
    `out` may be the residual or y itself."""
    if stream is not None:
        with _on(stream):
            return qmoe_block_norm(y, residual=residual, gate=gate, gating=gating,
                                   post_weight=post_weight, pre_weight=pre_weight,
                                   residual_scale=residual_scale, weight_offset=weight_offset,
                                   eps=eps, out=out, normed=normed)
    return (operators._module or _native()).block_norm(
        y, residual, gate, gating, post_weight, pre_weight, residual_scale, weight_offset, eps, out,
        normed)


def qmoe_block_norm_backward(dout: Optional[torch.Tensor], dnormed: Optional[torch.Tensor],
                             y: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                             residual: bool = True, gate: Optional[torch.Tensor] = None,
                             gating: int = QMOE_GATING_LINEAR,
                             post_weight: Optional[torch.Tensor] = None,
                             pre_weight: Optional[torch.Tensor] = None,
                             post_rstd: Optional[torch.Tensor] = None,
                             pre_rstd: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                             weight_offset: float = 0.0,
                             gate_grad_dtype: Optional[torch.dtype] = None, stream=None):
    """Gradients of qmoe_block_norm from those of its out and normed (dnormed with pre_weight and
    only then), for what it was given and returned (out: needed with pre_weight; None where it
    would be y); residual: whether its gradient is wanted.  Returns (dy, dresidual, dgate,
    dpost_weight, dpre_weight), None for what there is not; the weights' and a token's or channel's
    gate's gradients are fp32, a full gate's is of y's dtype, or of the gate's own where
    gate_grad_dtype says so (as autograd has it)."""
    if stream is not None:
        with _on(stream):
            return qmoe_block_norm_backward(
                dout, dnormed, y, out=out, residual=residual, gate=gate, gating=gating,
                post_weight=post_weight, pre_weight=pre_weight, post_rstd=post_rstd,
                pre_rstd=pre_rstd, residual_scale=residual_scale, weight_offset=weight_offset,
                gate_grad_dtype=gate_grad_dtype)
    own = gate_grad_dtype is not None and gate_grad_dtype != y.dtype
    if own and (gate is None or gate_grad_dtype != gate.dtype):
        raise ValueError(f"gate_grad_dtype: need y's or the gate's dtype, got {gate_grad_dtype}")
    return (operators._module or _native()).block_norm_backward(
        dout, dnormed, y, out, gate, gating, post_weight, pre_weight, residual_scale, weight_offset,
        post_rstd, pre_rstd, residual, True, True, True, own)


# ---------------------------------------------------------------- checkpoints in 8 bits
def qmoe_checkpoint8(x: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, stream=None):
    """x [M][C] in 8 bits: (codes int8 [M][C], scales uint8 [M][ceil(C / 32)]), x = code *
    2^(scale - 127) to within half a step of each block of 32 columns; a block with an infinity or
    NaN has scale 255."""
    if stream is not None:
        with _on(stream):
            return qmoe_checkpoint8(x, codes=codes, scales=scales)
    return (operators._module or _native()).checkpoint8(x, codes, scales)


def qmoe_checkpoint8_restore(codes: torch.Tensor, scales: torch.Tensor,
                             dtype: torch.dtype = torch.bfloat16, *,
                             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values [M][C] that codes and scales stand for (NaN for blocks of scale 255)."""
    if stream is not None:
        with _on(stream):
            return qmoe_checkpoint8_restore(codes, scales, dtype, out=out)
    like = out if out is not None and out.dtype == dtype else torch.empty(0, dtype=dtype)
    return (operators._module or _native()).checkpoint8_restore(codes, scales, like, out)


# --------------------------------------------------------------- gated feed-forward block
def qmoe_gated_ffn_workspace_size(M: int, H: int, I: int) -> int:
    return qmoe.lib().qmoe_gated_ffn_workspace_size(M, H, I)


def qmoe_gated_ffn_backward_workspace_size(M: int, H: int, I: int, checkpoint: int = 16) -> int:
    return qmoe.lib().qmoe_gated_ffn_backward_workspace_size(M, H, I, checkpoint)


def _bits(checkpoint: int) -> int:
    if checkpoint not in (8, 16):
        raise ValueError(f"checkpoint: need 16 or 8 bits, got {checkpoint}")
    return checkpoint


def qmoe_gated_ffn(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, *,
                   activation: int = QMOE_ACT_SILU, limit: float = math.inf, checkpoint: int = 16,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """out = (act(min(g, limit)) clamp(u, -limit, limit)) w2^T with [u | g] = x w13^T: x [M][H],
    w13 [2I][H] (rows 0..I-1 up, I..2I-1 gate, as the layer's), w2 [H][I], bf16 or fp16; out [M][H].
    checkpoint: bits in which a call that autograd has to know of keeps x, u and g for its
    backward pass (8: qmoe_checkpoint8's format)."""
    if stream is not None:
        with _on(stream):
            return qmoe_gated_ffn(x, w13, w2, activation=activation, limit=limit,
                                  checkpoint=checkpoint, out=out, workspace=workspace)
    return (operators._module or _native()).gated_ffn(x, w13, w2, activation, limit, 0, out,
                                                      workspace, _bits(checkpoint))


def qmoe_gated_ffn_saved(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, *,
                         activation: int = QMOE_ACT_SILU, limit: float = math.inf,
                         checkpoint: int = 16, out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """qmoe_gated_ffn that also returns what its backward pass needs: (out, saved).  checkpoint 16:
    saved = (u beside g [M][2I],), and x itself is needed too; 8: (codes and scales of u beside
    g, codes and scales of x), without x.  The backward pass is the caller's
    (qmoe_gated_ffn_backward): outside torch.no_grad(), on tensors that require a gradient, a
    gradient that comes to out raises."""
    if stream is not None:
        with _on(stream):
            return qmoe_gated_ffn_saved(x, w13, w2, activation=activation, limit=limit,
                                        checkpoint=checkpoint, out=out, workspace=workspace)
    native = operators._module or _native()
    out, kept, scales = native.gated_ffn(x, w13, w2, activation, limit, _bits(checkpoint), out,
                                         workspace, 0)
    if checkpoint == 16:
        return out, (kept,)
    return out, (kept, scales, *native.checkpoint8(x, None, None))


def qmoe_gated_ffn_backward(dout: torch.Tensor, x: Optional[torch.Tensor], w13: torch.Tensor,
                            w2: torch.Tensor, saved, *, activation: int = QMOE_ACT_SILU,
                            limit: float = math.inf, workspace: Optional[torch.Tensor] = None,
                            stream=None):
    """Gradients (dx [M][H], dw13 [2I][H], dw2 [H][I]) of qmoe_gated_ffn from that of its out and
    what qmoe_gated_ffn_saved returned, for the same weights, activation and limit (x: not read
    where it was saved in 8 bits)."""
    if stream is not None:
        with _on(stream):
            return qmoe_gated_ffn_backward(dout, x, w13, w2, saved, activation=activation,
                                           limit=limit, workspace=workspace)
    if len(saved) == 1:
        kept, scales, held, held_scales = saved[0], None, x, None
    elif len(saved) == 4:
        kept, scales, held, held_scales = saved
    else:
        raise ValueError("saved: need what qmoe_gated_ffn_saved returned")
    return (operators._module or _native()).gated_ffn_backward(
        dout, held, held_scales, w13, w2, kept, scales, activation, limit, True, True, True,
        workspace)
