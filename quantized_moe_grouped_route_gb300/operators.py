"""Operators around the MoE layer (ctypes binding of the same-named C-ABI calls): the expert
gate, tokens in expert order and back with their gradients, and a projection with
per-request low-rank adapters.

Activations are CUDA tensors of bf16, fp16 or fp32 whose rows may lie apart (stride of the
last dimension 1); outputs are contiguous and allocated unless given.  Calls run on
``stream`` (default: the current stream) and never synchronise.  A call's inputs must be
ready on that stream; what it allocates belongs to that stream.
"""

from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import qmoe
from .qmoe import _check

QMOE_DTYPE_BF16 = 0
QMOE_DTYPE_FP16 = 1
QMOE_DTYPE_FP32 = 2
QMOE_GATE_SOFTMAX = 0
QMOE_GATE_SIGMOID = 1

_DTYPES = {torch.bfloat16: QMOE_DTYPE_BF16, torch.float16: QMOE_DTYPE_FP16,
           torch.float32: QMOE_DTYPE_FP32}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _on(stream):
    """(stream handle, context in which to allocate what the call needs)."""
    if stream is None:
        return torch.cuda.current_stream().cuda_stream, contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return stream.cuda_stream, torch.cuda.stream(stream)


def _rows(t: torch.Tensor, name: str, shape=None) -> int:
    """Checks a matrix of activation rows and returns its row stride in elements (0: the
    same row throughout, as an expanded gradient has it)."""
    if t.dtype not in _DTYPES or t.dim() != 2:
        raise ValueError(f"{name}: need a matrix of bf16, fp16 or fp32, got {t.dtype} "
                         f"{tuple(t.shape)}")
    _here(t, name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")
    n, width = t.shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be next to each other")
    return t.stride(0) if n > 1 else width


def _here(t: torch.Tensor, name: str):
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: need a tensor on the current CUDA device, got {t.device}")


def _dense(t: torch.Tensor, dtype, name: str, shape=None):
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous tensor of {dtype}, got {t.dtype}")
    _here(t, name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")


def _same(a: torch.Tensor, b: torch.Tensor, names: str):
    if a.dtype != b.dtype:
        raise ValueError(f"{names}: need one dtype, got {a.dtype} and {b.dtype}")


def _out(t: Optional[torch.Tensor], shape, dtype, device, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dense(t, dtype, name, shape)
    return t


def _space(t: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if t is None:
        return torch.empty(max(nbytes, 256), dtype=_U8, device=device)
    _dense(t, _U8, "workspace")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


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
    ld = _rows(logits, "logits")
    M, E = logits.shape
    if bias is not None:
        _dense(bias, _F32, "bias", (E,))
    handle, where = _on(stream)
    with where:
        ids = _out(topk_ids, (M, top_k), _I32, logits.device, "topk_ids")
        weights = _out(topk_weights, (M, top_k), _F32, logits.device, "topk_weights")
    _check("moe_gate", qmoe.lib().moe_gate(
        logits.data_ptr(), _DTYPES[logits.dtype], ld, M, E, top_k, scoring, _ptr(bias), n_group,
        topk_group, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), handle))
    return ids, weights


def moe_gate_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *,
                      scoring: int = QMOE_GATE_SOFTMAX, renormalize: bool = True,
                      scale: float = 1.0, dlogits: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Gradient of the logits [M][E] from the gradient of moe_gate's weights, for the ids
    it returned and the same scoring, renormalize and scale."""
    ld = _rows(logits, "logits")
    M, E = logits.shape
    _dense(topk_ids, _I32, "topk_ids", (M, topk_ids.shape[-1]))
    _dense(dweights, _F32, "dweights", topk_ids.shape)
    handle, where = _on(stream)
    with where:
        dlogits = _out(dlogits, (M, E), logits.dtype, logits.device, "dlogits")
    _check("moe_gate_backward", qmoe.lib().moe_gate_backward(
        dweights.data_ptr(), logits.data_ptr(), _DTYPES[logits.dtype], ld, topk_ids.data_ptr(), M,
        E, topk_ids.shape[1], scoring, 1 if renormalize else 0, scale, dlogits.data_ptr(),
        handle))
    return dlogits


# --------------------------------------------------------------- tokens by expert
def qmoe_sort_workspace_size(M: int, top_k: int, E: int) -> int:
    return qmoe.lib().qmoe_sort_workspace_size(M, top_k, E)


def moe_sort_tokens(x: torch.Tensor, topk_ids: torch.Tensor, E: int, *,
                    xs: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """The rows of x [M][H] that the pairs of topk_ids int32 [M][top_k] route, in expert
    order: (xs [M*top_k][H], offsets [E+1], sorted_pair [M*top_k], pair_pos [M][top_k]),
    the tables as moe_route defines them; rows of xs past offsets[E] are zeros."""
    ldx = _rows(x, "x")
    M, H = x.shape
    _dense(topk_ids, _I32, "topk_ids", (M, topk_ids.shape[-1]))
    top_k = topk_ids.shape[1]
    dev = x.device
    L = qmoe.lib()
    need = L.qmoe_sort_workspace_size(M, top_k, E)
    handle, where = _on(stream)
    with where:
        xs = _out(xs, (M * top_k, H), x.dtype, dev, "xs")
        make = torch.empty if M else torch.zeros  # no tokens: every offset is 0
        offsets = make(max(E, 0) + 1, dtype=_I32, device=dev)
        sorted_pair = torch.empty(M * top_k, dtype=_I32, device=dev)
        pair_pos = torch.empty(M, top_k, dtype=_I32, device=dev)
        workspace = _space(workspace, need, dev)
    _check("moe_sort_tokens", L.moe_sort_tokens(
        x.data_ptr(), _DTYPES[x.dtype], ldx, topk_ids.data_ptr(), M, H, top_k, E, xs.data_ptr(),
        offsets.data_ptr(), sorted_pair.data_ptr(), pair_pos.data_ptr(), workspace.data_ptr(),
        workspace.numel(), handle))
    return xs, offsets, sorted_pair, pair_pos


def moe_sort_tokens_backward(dxs: torch.Tensor, pair_pos: torch.Tensor, *,
                             dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of x [M][H] from the gradient of moe_sort_tokens' xs: each token's routed
    rows added in slot order."""
    _dense(pair_pos, _I32, "pair_pos", (pair_pos.shape[0], pair_pos.shape[-1]))
    M, top_k = pair_pos.shape
    H = dxs.shape[-1]
    ld = _rows(dxs, "dxs", (M * top_k, H))
    handle, where = _on(stream)
    with where:
        dx = _out(dx, (M, H), dxs.dtype, dxs.device, "dx")
    _check("moe_sort_tokens_backward", qmoe.lib().moe_sort_tokens_backward(
        dxs.data_ptr(), _DTYPES[dxs.dtype], ld, pair_pos.data_ptr(), M, H, top_k, dx.data_ptr(),
        handle))
    return dx


def moe_unsort_tokens(y: torch.Tensor, pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expert outputs y [M*top_k][H] back in token order: out[m] = sum over the token's
    routed pairs of topk_weights[m][k] * y[pair_pos[m][k]], [M][H]."""
    _dense(pair_pos, _I32, "pair_pos", (pair_pos.shape[0], pair_pos.shape[-1]))
    M, top_k = pair_pos.shape
    _dense(topk_weights, _F32, "topk_weights", (M, top_k))
    H = y.shape[-1]
    ld = _rows(y, "y", (M * top_k, H))
    handle, where = _on(stream)
    with where:
        out = _out(out, (M, H), y.dtype, y.device, "out")
    _check("moe_unsort_tokens", qmoe.lib().moe_unsort_tokens(
        y.data_ptr(), _DTYPES[y.dtype], ld, pair_pos.data_ptr(), topk_weights.data_ptr(), M, H,
        top_k, out.data_ptr(), handle))
    return out


def moe_unsort_tokens_backward(dout: torch.Tensor, y: torch.Tensor, sorted_pair: torch.Tensor,
                               pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                               dy: Optional[torch.Tensor] = None,
                               dweights: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_unsort_tokens: (dy [M*top_k][H], dweights fp32 [M][top_k]); zeros
    for skipped pairs and for the rows past the routed ones."""
    _dense(pair_pos, _I32, "pair_pos", (pair_pos.shape[0], pair_pos.shape[-1]))
    M, top_k = pair_pos.shape
    _dense(sorted_pair, _I32, "sorted_pair", (M * top_k,))
    _dense(topk_weights, _F32, "topk_weights", (M, top_k))
    H = y.shape[-1]
    ldy = _rows(y, "y", (M * top_k, H))
    ldd = _rows(dout, "dout", (M, H))
    _same(dout, y, "dout, y")
    handle, where = _on(stream)
    with where:
        dy = _out(dy, (M * top_k, H), y.dtype, y.device, "dy")
        dweights = _out(dweights, (M, top_k), _F32, y.device, "dweights")
    _check("moe_unsort_tokens_backward", qmoe.lib().moe_unsort_tokens_backward(
        dout.data_ptr(), ldd, y.data_ptr(), ldy, _DTYPES[y.dtype], sorted_pair.data_ptr(),
        pair_pos.data_ptr(), topk_weights.data_ptr(), M, H, top_k, dy.data_ptr(),
        dweights.data_ptr(), handle))
    return dy, dweights


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
    ldx = _rows(x, "x")
    dt = x.dtype
    M, K = x.shape
    if lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("lora_a, lora_b: need [L][R][K] and [L][N][R]")
    L, R = lora_a.shape[:2]
    N = lora_b.shape[1]
    _dense(lora_a, dt, "lora_a", (L, R, K))
    _dense(lora_b, dt, "lora_b", (L, N, R))
    if w is not None:
        _dense(w, dt, "w", (N, K))
    _dense(adapter_ids, _I32, "adapter_ids", (M,))
    _dense(scales, _F32, "scales", (L,))
    ldb = 0
    if base is not None:
        ldb = _rows(base, "base", (M, N))
        _same(x, base, "x, base")
    lib = qmoe.lib()
    need = lib.qmoe_lora_workspace_size(M, K, N, R, L)
    handle, where = _on(stream)
    with where:
        out = _out(out, (M, N), dt, x.device, "out")
        workspace = _space(workspace, need, x.device)
    _check("qmoe_lora_linear", lib.qmoe_lora_linear(
        x.data_ptr(), _DTYPES[dt], ldx, _ptr(w), lora_a.data_ptr(), lora_b.data_ptr(),
        adapter_ids.data_ptr(), scales.data_ptr(), _ptr(base), ldb, out.data_ptr(), M, K, N, R, L,
        workspace.data_ptr(), workspace.numel(), handle))
    return out
