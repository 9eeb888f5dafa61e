"""Operators around the MoE layer (binding of the same-named C-ABI calls): the expert gate,
tokens in expert order and back with their gradients, and a projection with per-request
low-rank adapters.

Activations are CUDA tensors of bf16, fp16 or fp32 whose rows may lie apart (stride of the
last dimension 1); outputs are contiguous and allocated unless given.  Calls run on
``stream`` (default: the current stream) and never synchronise.  A call's inputs must be
ready on that stream; what it allocates belongs to that stream (tensors that another stream
uses too need record_stream, as for torch's own calls).  A tensor that does not fit
raises ValueError, a refusal of the library QmoeError.  What a kernel finds (ids out of range,
an expired wait) is in the error word at the start of a given workspace (qmoe_read_error), of
calls that were given none in qmoe_default_read_error.

Autograd: moe_gate, moe_sort_tokens and moe_unsort_tokens on tensors that require a gradient
are nodes of its graph, whose backward is the *_backward call of the same name (those calls
have no derivative of their own); qmoe_lora_linear has none, and a gradient that comes to it
raises NotImplementedError.  Such a call takes no outputs to write into.  An output that is given
counts as changed in place (a node that has kept it raises) and may itself require a gradient under
torch.no_grad() alone.  None has a derivative in forward mode: a tensor that carries a tangent
raises NotImplementedError, grad mode or not.

Checks, allocations and the call itself are compiled (csrc/binding.cpp, qmoe_torch.so).
"""

from __future__ import annotations

import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import qmoe
from .qmoe import QmoeError

QMOE_DTYPE_BF16 = 0
QMOE_DTYPE_FP16 = 1
QMOE_DTYPE_FP32 = 2
QMOE_GATE_SOFTMAX = 0
QMOE_GATE_SIGMOID = 1

BINDING_PATH = os.path.join(os.path.dirname(qmoe.LIB_PATH), "qmoe_torch.so")
_module = None


def _native():
    """The compiled part (raises if it has not been built)."""
    global _module
    if _module is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"qmoe_torch.so is missing at {BINDING_PATH}: run "
                               "`python -m quantized_moe_grouped_route_gb300.build`")
        qmoe.lib()
        loader = importlib.machinery.ExtensionFileLoader("qmoe_torch", BINDING_PATH)
        spec = importlib.util.spec_from_loader("qmoe_torch", loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.set_error(QmoeError)
        module.set_graph(_graph)
        _module = module
    return _module


def _on(stream):
    """A context in which the given stream is current."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def qmoe_default_read_error(stream=None):
    """(return code, flags) of the last moe_sort_tokens, qmoe_lora_linear, qmoe_gated_ffn and
    qmoe_gated_ffn_backward calls on the current device that were given no workspace, together;
    their workspaces are kept until the next such call (a gated block's of more than 1 MiB is not,
    its error word alone).  Synchronises the stream (default: the current one), on which, or before
    which, those calls were made."""
    rc, flags = qmoe.QMOE_OK, 0
    for workspace in (_module or _native()).default_workspaces():
        one, found = qmoe.qmoe_read_error(workspace, stream)
        rc, flags = rc or one, flags | found
    return rc, flags


# ------------------------------------------------------------------------ autograd
def _rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the library takes rows: their elements next to each other."""
    apart = t.stride(0) if t.size(0) > 1 else t.size(1)
    fits = (t.size(1) < 2 or t.stride(1) == 1) and (apart == 0 or apart >= t.size(1))
    return t if fits else t.contiguous()


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, scoring, bias, n_group, topk_group, renormalize, scale, ids,
                weights):
        ids, weights = _native().gate(logits, top_k, scoring, bias, n_group, topk_group,
                                      renormalize, scale, ids, weights)
        ctx.save_for_backward(logits, ids)
        ctx.how = (scoring, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dweights):
        logits, ids = ctx.saved_tensors
        dlogits = _native().gate_backward(dweights.contiguous(), logits, ids, *ctx.how, None)
        return (dlogits,) + 9 * (None,)


class _SortTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, E, xs, workspace):
        xs, *tables = _native().sort_tokens(x, ids, E, xs, workspace)
        ctx.save_for_backward(tables[2])
        ctx.mark_non_differentiable(*tables)
        return (xs, *tables)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs, *_):
        dx = _native().sort_tokens_backward(_rows(dxs), *ctx.saved_tensors, None)
        return (dx,) + 4 * (None,)


class _UnsortTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, pair_pos, weights, out):
        ctx.save_for_backward(y, pair_pos, weights)
        return _native().unsort_tokens(y, pair_pos, weights, out)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, pair_pos, weights = ctx.saved_tensors
        # sorted_pair from its inverse; pairs without a row write past the end
        P = pair_pos.numel()
        pos = pair_pos.reshape(-1).long()
        pos = torch.where((pos >= 0) & (pos < P), pos, P)
        pairs = torch.arange(P, dtype=torch.int32, device=y.device)
        sorted_pair = pairs.new_full((P + 1,), -1).scatter_(0, pos, pairs)[:P]
        dy, dweights = _native().unsort_tokens_backward(_rows(dout), y, sorted_pair, pair_pos,
                                                        weights, None, None)
        return dy, None, dweights, None


class _LoraLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *args):
        return _native().lora_linear(*args)

    @staticmethod
    def backward(ctx, _):
        raise NotImplementedError("qmoe_lora_linear has no gradient: call it under torch.no_grad() "
                                  "or on detached tensors")


# of each call the node, and which of its arguments are outputs
_NODES = {"gate": (_Gate, (8, 9)), "sort_tokens": (_SortTokens, (3,)),
          "unsort_tokens": (_UnsortTokens, (3,)), "lora_linear": (_LoraLinear, (7,))}


def _graph(name, *args):
    """A call on tensors that require a gradient (the compiled part hands it over)."""
    node, outputs = _NODES[name]
    if any(args[i] is not None for i in outputs):
        raise ValueError("a call on tensors that require a gradient returns new tensors: no "
                         "output to write into can be given (or call it under torch.no_grad())")
    return node.apply(*args)


# ---------------------------------------------------------------------------- gate
def moe_gate(logits: torch.Tensor, top_k: int, *, scoring: int = QMOE_GATE_SOFTMAX,
             bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
             renormalize: bool = True, scale: float = 1.0,
             topk_ids: Optional[torch.Tensor] = None,
             topk_weights: Optional[torch.Tensor] = None, stream=None):
    """Each token's experts and routing weights from the router's logits [M][E]:
    (topk_ids int32 [M][top_k], topk_weights fp32 [M][top_k]), ready for moe_route and the
    layer.  scoring: softmax, or sigmoid with an optional selection bias fp32 [E]; experts
    in n_group runs of which the topk_group best stay; logits of -infinity mask experts,
    and slots left over get id -1 and weight 0."""
    if stream is not None:
        with _on(stream):
            return moe_gate(logits, top_k, scoring=scoring, bias=bias, n_group=n_group,
                            topk_group=topk_group, renormalize=renormalize, scale=scale,
                            topk_ids=topk_ids, topk_weights=topk_weights)
    return (_module or _native()).gate(logits, top_k, scoring, bias, n_group, topk_group,
                                       renormalize, scale, topk_ids, topk_weights)


def moe_gate_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *,
                      scoring: int = QMOE_GATE_SOFTMAX, renormalize: bool = True,
                      scale: float = 1.0, dlogits: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Gradient of the logits [M][E] from the gradient of moe_gate's weights, for the ids
    it returned and the same scoring, renormalize and scale."""
    if stream is not None:
        with _on(stream):
            return moe_gate_backward(dweights, logits, topk_ids, scoring=scoring,
                                     renormalize=renormalize, scale=scale, dlogits=dlogits)
    return (_module or _native()).gate_backward(dweights, logits, topk_ids, scoring, renormalize,
                                                scale, dlogits)


# --------------------------------------------------------------- tokens by expert
def qmoe_sort_workspace_size(M: int, top_k: int, E: int) -> int:
    return qmoe.lib().qmoe_sort_workspace_size(M, top_k, E)


def moe_sort_tokens(x: torch.Tensor, topk_ids: torch.Tensor, E: int, *,
                    xs: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """The rows of x [M][H] that the pairs of topk_ids int32 [M][top_k] route, in expert
    order: (xs [M*top_k][H], offsets [E+1], sorted_pair [M*top_k], pair_pos [M][top_k]),
    the tables as moe_route defines them; rows of xs past offsets[E] are zeros."""
    if stream is not None:
        with _on(stream):
            return moe_sort_tokens(x, topk_ids, E, xs=xs, workspace=workspace)
    return (_module or _native()).sort_tokens(x, topk_ids, E, xs, workspace)


def moe_sort_tokens_backward(dxs: torch.Tensor, pair_pos: torch.Tensor, *,
                             dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of x [M][H] from the gradient of moe_sort_tokens' xs: each token's routed
    rows added in slot order."""
    if stream is not None:
        with _on(stream):
            return moe_sort_tokens_backward(dxs, pair_pos, dx=dx)
    return (_module or _native()).sort_tokens_backward(dxs, pair_pos, dx)


def moe_unsort_tokens(y: torch.Tensor, pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expert outputs y [M*top_k][H] back in token order: out[m] = sum over the token's
    routed pairs of topk_weights[m][k] * y[pair_pos[m][k]], [M][H]."""
    if stream is not None:
        with _on(stream):
            return moe_unsort_tokens(y, pair_pos, topk_weights, out=out)
    return (_module or _native()).unsort_tokens(y, pair_pos, topk_weights, out)


def moe_unsort_tokens_backward(dout: torch.Tensor, y: torch.Tensor, sorted_pair: torch.Tensor,
                               pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                               dy: Optional[torch.Tensor] = None,
                               dweights: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_unsort_tokens: (dy [M*top_k][H], dweights fp32 [M][top_k]); zeros
    for skipped pairs and for the rows past the routed ones."""
    if stream is not None:
        with _on(stream):
            return moe_unsort_tokens_backward(dout, y, sorted_pair, pair_pos, topk_weights, dy=dy,
                                              dweights=dweights)
    return (_module or _native()).unsort_tokens_backward(dout, y, sorted_pair, pair_pos,
                                                         topk_weights, dy, dweights)


# ------------------------------------------------------------ adapters of many requests
def qmoe_lora_workspace_size(M: int, K: int, N: int, R: int, L: int) -> int:
    return qmoe.lib().qmoe_lora_workspace_size(M, K, N, R, L)


def qmoe_lora_linear(x: torch.Tensor, w: Optional[torch.Tensor], lora_a: torch.Tensor,
                     lora_b: torch.Tensor, adapter_ids: torch.Tensor, scales: torch.Tensor, *,
                     base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[m] = base[m] + x[m] w^T + scales[a] (x[m] A[a]^T) B[a]^T with a = adapter_ids[m]
    (negative: no adapter).  x [M][K] bf16 or fp16, w [N][K] or None, lora_a [L][R][K],
    lora_b [L][N][R], adapter_ids int32 [M], scales fp32 [L], base [M][N] or None (may be
    `out`); out [M][N]."""
    if stream is not None:
        with _on(stream):
            return qmoe_lora_linear(x, w, lora_a, lora_b, adapter_ids, scales, base=base, out=out,
                                    workspace=workspace)
    return (_module or _native()).lora_linear(x, w, lora_a, lora_b, adapter_ids, scales, base, out,
                                              workspace)
