"""Operators around the MoE layer (ctypes binding of the same-named C-ABI calls): the expert
gate, tokens in expert order and back with their gradients, and a projection with
per-request low-rank adapters.

Activations are CUDA tensors of bf16, fp16 or fp32 whose rows may lie apart (stride of the
last dimension 1); outputs are contiguous and allocated unless given.  Calls run on
``stream`` (default: the current stream) and never synchronise.  A call's inputs must be
ready on that stream; what it allocates belongs to that stream.

The smallest calls are over on the GPU sooner than Python can issue them, so the argument
checks below are written for few interpreter steps: on the host of a GB300 the decode gate
(M = 16, E = 256) took 16.8 us a call with the checks in helpers of their own and
torch.cuda.current_stream(), of which the C call with its launch is 3.6 us.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import qmoe
from .qmoe import QmoeError

QMOE_DTYPE_BF16 = 0
QMOE_DTYPE_FP16 = 1
QMOE_DTYPE_FP32 = 2
QMOE_GATE_SOFTMAX = 0
QMOE_GATE_SIGMOID = 1

_DTYPES = {torch.bfloat16: QMOE_DTYPE_BF16, torch.float16: QMOE_DTYPE_FP16,
           torch.float32: QMOE_DTYPE_FP32}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream


def _device() -> int:
    """Index of the current device (every tensor of a call lies on it)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


class _On:
    """Makes a given stream current, so that allocations inside belong to it."""

    def __init__(self, stream):
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        self._context = torch.cuda.stream(stream)

    def __enter__(self):
        self._context.__enter__()

    def __exit__(self, *exc):
        return self._context.__exit__(*exc)


def _rows(t: torch.Tensor, name: str, dev: int, shape=None) -> int:
    """Checks a matrix of activation rows and returns its row stride in elements (0: the
    same row throughout, as an expanded gradient has it)."""
    if t.dtype not in _DTYPES or t.dim() != 2:
        raise ValueError(f"{name}: need a matrix of bf16, fp16 or fp32, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name}: need a tensor on the current CUDA device, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, one = t.stride()
    n, width = t.shape
    if one != 1 and width > 1:
        raise ValueError(f"{name}: the elements of a row must be next to each other")
    return ld if n > 1 else width


def _dense(t: torch.Tensor, dtype, name: str, dev: int, shape=None):
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous tensor of {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name}: need a tensor on the current CUDA device, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")


def _pairs(t: torch.Tensor, name: str, dev: int):
    """(M, top_k) of an int32 [M][top_k] table."""
    if t.dim() != 2:
        raise ValueError(f"{name}: need [M][top_k], got {tuple(t.shape)}")
    _dense(t, _I32, name, dev)
    return t.shape


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
        with _On(stream):
            return moe_gate(logits, top_k, scoring=scoring, bias=bias, n_group=n_group,
                            topk_group=topk_group, renormalize=renormalize, scale=scale,
                            topk_ids=topk_ids, topk_weights=topk_weights)
    dev = _device()
    ld = _rows(logits, "logits", dev)
    M, E = logits.shape
    pb = None
    if bias is not None:
        _dense(bias, _F32, "bias", dev, (E,))
        pb = bias.data_ptr()
    shape = (M, top_k)
    if topk_ids is None:
        topk_ids = _empty(shape, dtype=_I32, device=logits.device)
    else:
        _dense(topk_ids, _I32, "topk_ids", dev, shape)
    if topk_weights is None:
        topk_weights = _empty(shape, dtype=_F32, device=logits.device)
    else:
        _dense(topk_weights, _F32, "topk_weights", dev, shape)
    rc = qmoe.lib().moe_gate(
        logits.data_ptr(), _DTYPES[logits.dtype], ld, M, E, top_k, scoring, pb, n_group,
        topk_group, 1 if renormalize else 0, scale, topk_ids.data_ptr(),
        topk_weights.data_ptr(), _raw_stream(dev))
    if rc:
        raise QmoeError("moe_gate", rc)
    return topk_ids, topk_weights


def moe_gate_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *,
                      scoring: int = QMOE_GATE_SOFTMAX, renormalize: bool = True,
                      scale: float = 1.0, dlogits: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Gradient of the logits [M][E] from the gradient of moe_gate's weights, for the ids
    it returned and the same scoring, renormalize and scale."""
    if stream is not None:
        with _On(stream):
            return moe_gate_backward(dweights, logits, topk_ids, scoring=scoring,
                                     renormalize=renormalize, scale=scale, dlogits=dlogits)
    dev = _device()
    ld = _rows(logits, "logits", dev)
    M, E = logits.shape
    top_k = topk_ids.shape[-1]
    _dense(topk_ids, _I32, "topk_ids", dev, (M, top_k))
    _dense(dweights, _F32, "dweights", dev, (M, top_k))
    if dlogits is None:
        dlogits = _empty((M, E), dtype=logits.dtype, device=logits.device)
    else:
        _dense(dlogits, logits.dtype, "dlogits", dev, (M, E))
    rc = qmoe.lib().moe_gate_backward(
        dweights.data_ptr(), logits.data_ptr(), _DTYPES[logits.dtype], ld, topk_ids.data_ptr(), M,
        E, top_k, scoring, 1 if renormalize else 0, scale, dlogits.data_ptr(), _raw_stream(dev))
    if rc:
        raise QmoeError("moe_gate_backward", rc)
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
    if stream is not None:
        with _On(stream):
            return moe_sort_tokens(x, topk_ids, E, xs=xs, workspace=workspace)
    dev = _device()
    ldx = _rows(x, "x", dev)
    M, H = x.shape
    top_k = topk_ids.shape[-1]
    _dense(topk_ids, _I32, "topk_ids", dev, (M, top_k))
    device, P = x.device, M * top_k
    lib = qmoe.lib()
    if xs is None:
        xs = _empty((P, H), dtype=x.dtype, device=device)
    else:
        _dense(xs, x.dtype, "xs", dev, (P, H))
    if workspace is None:
        workspace = _empty(lib.qmoe_sort_workspace_size(M, top_k, E), dtype=_U8, device=device)
    else:
        _dense(workspace, _U8, "workspace", dev)
    if E < 1:
        raise QmoeError("moe_sort_tokens", qmoe.QMOE_ERR_SHAPE)
    make = _empty if M else torch.zeros  # no tokens: every offset is 0
    offsets = make(E + 1, dtype=_I32, device=device)
    sorted_pair = _empty(P, dtype=_I32, device=device)
    pair_pos = _empty((M, top_k), dtype=_I32, device=device)
    rc = lib.moe_sort_tokens(
        x.data_ptr(), _DTYPES[x.dtype], ldx, topk_ids.data_ptr(), M, H, top_k, E, xs.data_ptr(),
        offsets.data_ptr(), sorted_pair.data_ptr(), pair_pos.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _raw_stream(dev))
    if rc:
        raise QmoeError("moe_sort_tokens", rc)
    return xs, offsets, sorted_pair, pair_pos


def moe_sort_tokens_backward(dxs: torch.Tensor, pair_pos: torch.Tensor, *,
                             dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of x [M][H] from the gradient of moe_sort_tokens' xs: each token's routed
    rows added in slot order."""
    if stream is not None:
        with _On(stream):
            return moe_sort_tokens_backward(dxs, pair_pos, dx=dx)
    dev = _device()
    M, top_k = _pairs(pair_pos, "pair_pos", dev)
    H = dxs.shape[-1]
    ld = _rows(dxs, "dxs", dev, (M * top_k, H))
    if dx is None:
        dx = _empty((M, H), dtype=dxs.dtype, device=dxs.device)
    else:
        _dense(dx, dxs.dtype, "dx", dev, (M, H))
    rc = qmoe.lib().moe_sort_tokens_backward(
        dxs.data_ptr(), _DTYPES[dxs.dtype], ld, pair_pos.data_ptr(), M, H, top_k, dx.data_ptr(),
        _raw_stream(dev))
    if rc:
        raise QmoeError("moe_sort_tokens_backward", rc)
    return dx


def moe_unsort_tokens(y: torch.Tensor, pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expert outputs y [M*top_k][H] back in token order: out[m] = sum over the token's
    routed pairs of topk_weights[m][k] * y[pair_pos[m][k]], [M][H]."""
    if stream is not None:
        with _On(stream):
            return moe_unsort_tokens(y, pair_pos, topk_weights, out=out)
    dev = _device()
    M, top_k = _pairs(pair_pos, "pair_pos", dev)
    _dense(topk_weights, _F32, "topk_weights", dev, (M, top_k))
    H = y.shape[-1]
    ld = _rows(y, "y", dev, (M * top_k, H))
    if out is None:
        out = _empty((M, H), dtype=y.dtype, device=y.device)
    else:
        _dense(out, y.dtype, "out", dev, (M, H))
    rc = qmoe.lib().moe_unsort_tokens(
        y.data_ptr(), _DTYPES[y.dtype], ld, pair_pos.data_ptr(), topk_weights.data_ptr(), M, H,
        top_k, out.data_ptr(), _raw_stream(dev))
    if rc:
        raise QmoeError("moe_unsort_tokens", rc)
    return out


def moe_unsort_tokens_backward(dout: torch.Tensor, y: torch.Tensor, sorted_pair: torch.Tensor,
                               pair_pos: torch.Tensor, topk_weights: torch.Tensor, *,
                               dy: Optional[torch.Tensor] = None,
                               dweights: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_unsort_tokens: (dy [M*top_k][H], dweights fp32 [M][top_k]); zeros
    for skipped pairs and for the rows past the routed ones."""
    if stream is not None:
        with _On(stream):
            return moe_unsort_tokens_backward(dout, y, sorted_pair, pair_pos, topk_weights, dy=dy,
                                              dweights=dweights)
    dev = _device()
    M, top_k = _pairs(pair_pos, "pair_pos", dev)
    P, H = M * top_k, y.shape[-1]
    _dense(sorted_pair, _I32, "sorted_pair", dev, (P,))
    _dense(topk_weights, _F32, "topk_weights", dev, (M, top_k))
    ldy = _rows(y, "y", dev, (P, H))
    ldd = _rows(dout, "dout", dev, (M, H))
    if dout.dtype != y.dtype:
        raise ValueError(f"dout, y: need one dtype, got {dout.dtype} and {y.dtype}")
    if dy is None:
        dy = _empty((P, H), dtype=y.dtype, device=y.device)
    else:
        _dense(dy, y.dtype, "dy", dev, (P, H))
    if dweights is None:
        dweights = _empty((M, top_k), dtype=_F32, device=y.device)
    else:
        _dense(dweights, _F32, "dweights", dev, (M, top_k))
    rc = qmoe.lib().moe_unsort_tokens_backward(
        dout.data_ptr(), ldd, y.data_ptr(), ldy, _DTYPES[y.dtype], sorted_pair.data_ptr(),
        pair_pos.data_ptr(), topk_weights.data_ptr(), M, H, top_k, dy.data_ptr(),
        dweights.data_ptr(), _raw_stream(dev))
    if rc:
        raise QmoeError("moe_unsort_tokens_backward", rc)
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
    if stream is not None:
        with _On(stream):
            return qmoe_lora_linear(x, w, lora_a, lora_b, adapter_ids, scales, base=base, out=out,
                                    workspace=workspace)
    dev = _device()
    ldx = _rows(x, "x", dev)
    dt = x.dtype
    M, K = x.shape
    if lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("lora_a, lora_b: need [L][R][K] and [L][N][R]")
    L, R, _ = lora_a.shape
    N = lora_b.shape[1]
    _dense(lora_a, dt, "lora_a", dev, (L, R, K))
    _dense(lora_b, dt, "lora_b", dev, (L, N, R))
    _dense(adapter_ids, _I32, "adapter_ids", dev, (M,))
    _dense(scales, _F32, "scales", dev, (L,))
    pw = pb = None
    ldb = 0
    if w is not None:
        _dense(w, dt, "w", dev, (N, K))
        pw = w.data_ptr()
    if base is not None:
        ldb = _rows(base, "base", dev, (M, N))
        if base.dtype != dt:
            raise ValueError(f"x, base: need one dtype, got {dt} and {base.dtype}")
        pb = base.data_ptr()
    lib = qmoe.lib()
    if out is None:
        out = _empty((M, N), dtype=dt, device=x.device)
    else:
        _dense(out, dt, "out", dev, (M, N))
    if workspace is None:
        workspace = _empty(lib.qmoe_lora_workspace_size(M, K, N, R, L), dtype=_U8,
                           device=x.device)
    else:
        _dense(workspace, _U8, "workspace", dev)
    rc = lib.qmoe_lora_linear(
        x.data_ptr(), _DTYPES[dt], ldx, pw, lora_a.data_ptr(), lora_b.data_ptr(),
        adapter_ids.data_ptr(), scales.data_ptr(), pb, ldb, out.data_ptr(), M, K, N, R, L,
        workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    if rc:
        raise QmoeError("qmoe_lora_linear", rc)
    return out
