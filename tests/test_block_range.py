"""The norms around a block and the gated feed-forward block where values, plans or rings leave what
small batches of normal numbers reach.  Bounds as in test_block_operators.py."""

import math

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe
from tests import test_block_operators as ops
from tests.test_block_operators import (ACTS, ROUND, U, _case, _ffn_grads, _ffn_inputs, _gen, _near,
                                        _norm_call, _norm_inputs, _rows)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- gates far from 0
def _norm_backward(c, s, out, dout, dn, post, pre, **kw):
    return q.qmoe_block_norm_backward(
        dout, dn, s["y"], out=out, residual=c["residual"], gate=s["gate"],
        gating=int(c["sigmoid"]), post_weight=s["post"], pre_weight=s["pre"], post_rstd=post,
        pre_rstd=pre, residual_scale=c["scale"], weight_offset=c["offset"], **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", ["token", "channel", "full"])
@pytest.mark.parametrize("M,H", [(40, 264), (3, 33), (2, 8200)])
def test_gradient_of_a_saturated_gate(M, H, form, dtype):
    """sigmoid(l) of l from -60 to 60: its slope is sigmoid(l) sigmoid(-l), which 1 - sigmoid(l) has
    no digits for past 17.  A sigmoid by exp and a division is within a few u, the slope a product of
    two; the terms' own errors are those of a gate of 1 (whose slope is 1), so they scale with it."""
    c = _case(M, H, dtype, gate=form, pre=False, sigmoid=True)
    s = _norm_inputs(c, 5)
    s["gate"] = torch.linspace(-60, 60, s["gate"].numel(), device="cuda").view_as(s["gate"]).to(dtype)
    out, _, post, pre = _norm_call(c, s)
    dout = _rows(_gen(1), M, H, dtype)
    got = _norm_backward(c, s, out, dout, None, post, pre)[2]
    l = s["gate"].double()
    slope = torch.sigmoid(l) * torch.sigmoid(-l)
    unit = s["y"].double() * post.double()[:, None] * s["post"].double()
    each = dout.double() * unit
    if form == "full":
        ref, bound = each * slope, 32 * U * each.abs() * slope
    else:
        dim, n = (1, H) if form == "token" else (0, M)
        ref = each.sum(dim, keepdim=True) * slope
        bound = (n + 32) * U * each.abs().sum(dim, keepdim=True) * slope
    k = got.dtype
    # (slopes of 60 are 2^-86, far above the least normal numbers)
    _near(got, ref, bound + ROUND[k] * (ref.abs() + bound), "dgate")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,pad", [(9, 256, 0), (33, 1001, 3), (2, 8200, 0), (400, 72, 0)])
def test_a_full_gate_of_fp32_gets_its_gradient_in_fp32(M, H, pad, dtype):
    """Values held in fp32 reach an fp32 gate unrounded: also those past fp16's largest number and
    under its least."""
    c = _case(M, H, dtype, gate="full", fp32=True, pre=False, pad=pad)
    s = _norm_inputs(c, 6)
    leaf = s["gate"].clone().requires_grad_(True)
    out, _, post, pre = _norm_call(c, dict(s, gate=leaf))
    dout = _rows(_gen(1), M, H, dtype, pad)
    dout[0], dout[1] = 60000.0, 2.0 ** -24  # times v: past 65504 and under 2^-24 in some columns
    out.backward(dout)
    v = s["y"].double() * post.double()[:, None] * s["post"].double()
    ref = dout.double() * v
    assert ref.abs().max() > 65504 and leaf.grad.dtype == torch.float32
    bound = 32 * U * ref.abs()
    _near(leaf.grad, ref, bound, "dgate")
    # the explicit call: in the activations' type, or the gate's by asking
    own = _norm_backward(c, s, out.detach(), dout, None, post, pre, gate_grad_dtype=torch.float32)
    assert torch.equal(own[2], leaf.grad)
    plain = _norm_backward(c, s, out.detach(), dout, None, post, pre)
    assert plain[2].dtype == dtype and torch.equal(plain[2], own[2].to(dtype))
    for a, b in zip(own, plain):
        assert a is own[2] or (a is None and b is None) or torch.equal(a, b)
    with pytest.raises(ValueError):
        _norm_backward(c, s, out.detach(), dout, None, post, pre, gate_grad_dtype=torch.float64)


# --------------------------------------------------------- pre-activations past fp16's range
@pytest.mark.parametrize("M,H", [(5, 64), (5, 4096), (200, 64), (700, 72)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_kept_values_past_fp16(M, H, kind):
    """g of -100000 closes its gate and u of 100000 stays finite times an h that is: the forward pass
    is finite, and so are the gradients.  A finite u or g that fp16 has not is kept as its largest."""
    I, dt = 520, torch.float16
    x, w13, w2 = _ffn_inputs(M, H, I, dt)
    x[:, 0] = 400.0
    w13[:, 0] = 0.0
    w13[I + 3, 0] = w13[I + 17, 0] = -250.0  # g = -100000: h = 0
    w13[9, 0], w13[I + 9] = 250.0, 0.0  # u = 100000, g = 0: h = 0 too, dg = u dh / 2
    w2[:, 9] *= 2.0 ** -12  # (so that fp16 has dg)
    how = dict(activation=ACTS[kind])
    out, (kept,) = q.qmoe_gated_ffn_saved(x, w13, w2, **how)
    assert torch.isfinite(out).all() and torch.isfinite(kept).all()
    ug = x.double() @ w13.double().t()
    want = ug.clamp(-65504, 65504)
    assert (kept[:, [9, I + 3, I + 17]].double() == want[:, [9, I + 3, I + 17]]).all()
    dout = _rows(_gen(M), M, H, dt)
    got = q.qmoe_gated_ffn_backward(dout, x, w13, w2, (kept,), **how)
    u, g = kept[:, :I].double(), kept[:, I:].double()
    ref = _ffn_grads(kind, math.inf, dout, x, w13, w2, u, g, dt)
    for name, t in zip(("dx", "dw13", "dw2"), got):
        r, bound = ref[name]
        fits = r.abs() + bound < 65504  # (what fp16 has)
        _near(torch.where(fits, t.double(), 0.0), torch.where(fits, r, 0.0), bound, name)
    # a true infinity stays one
    x[0, 0] = math.inf
    out, (kept,) = q.qmoe_gated_ffn_saved(x, w13, w2, **how)
    assert kept[0, 9] == math.inf and not torch.isfinite(out[0]).any()


# ------------------------------------------------------------- gates that are nearly closed
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations_of_closed_gates(kind, dtype):
    """Both activations are g sigmoid(k(g)).  exp's approximation is off by 2 + 1.173 |k| units in the
    last place (2^-23) and k by a few of its own, so the sigmoid is off by (8 + 4 |k|) 2^-23, below
    the rounding of what it enters for every k at which the result is a number of the type.  Weights
    and tokens are rows of the identity: out is h, and the gradient of w13 is [du | dg]."""
    n = 64
    eye = torch.eye(n, device="cuda", dtype=dtype)
    least = {"silu": (-80.0, -15.0), "gelu": (-9.0, -3.5)}[kind][dtype == torch.float16]
    gates = torch.linspace(least, 10.0, n * n, device="cuda").view(n, n).to(dtype)
    w13 = torch.cat([torch.full((n, n), 0.75, device="cuda", dtype=dtype), gates.t()])
    out, saved = q.qmoe_gated_ffn_saved(eye, w13, eye, activation=ACTS[kind])
    g, u = gates.double(), 0.75
    A, B = math.sqrt(2 / math.pi), 0.044715
    k, dk = (g, 1.0) if kind == "silu" else (2 * A * (g + B * g ** 3), 2 * A * (1 + 3 * B * g * g))
    p, left = torch.sigmoid(k), torch.sigmoid(-k)
    rel = (8 + 4 * k.abs()) * 2.0 ** -23
    r, tiny = ROUND[dtype], ops.TINY[dtype]
    h = g * p * u
    _near(out, h, rel * h.abs() + r * h.abs() * (1 + rel) + tiny, "h")
    _near(q.qmoe_gated_ffn(eye, w13, eye, activation=ACTS[kind]), h,
          rel * h.abs() + r * h.abs() * (1 + rel) + tiny, "h of a call that keeps nothing")
    dout = torch.full((n, n), 2.0, device="cuda", dtype=dtype)
    dug = q.qmoe_gated_ffn_backward(dout, eye, w13, eye, saved, activation=ACTS[kind])[1].t()
    du, dg = 2 * g * p, 2 * u * (p + g * p * left * dk)
    terms = 2 * u * (p + (g * p * left * dk).abs())
    _near(dug[:, :n], du, rel * du.abs() + r * du.abs() * (1 + rel) + tiny, "du")
    _near(dug[:, n:], dg, 2 * rel * terms + r * (dg.abs() + 2 * rel * terms) + tiny, "dg")


# ------------------------------------------------------ plans that only large sizes take
WIDE = (2310, 1032, 2056)  # every product in tiles of 256 columns, with odd ends of M, N and K


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8])
def test_gated_ffn_in_wide_tiles(bits, dtype):
    """All elements of the outputs and gradients, as of small batches."""
    kind, limit = ("silu", 1.0) if bits == 8 else ("gelu", math.inf)
    ops.test_gated_ffn_saved(*WIDE, kind, limit, dtype)
    ops.test_gated_ffn_backward(*WIDE, kind, limit, bits, dtype)
    if bits == 16:
        ops.test_gated_ffn(*WIDE, kind, limit, dtype)


@pytest.mark.parametrize("M,H,I", [(8200, 264, 264), (300, 264, 4112), (2310, 1032, 2056)])
def test_a_corner_tile_of_many_steps(M, H, I):
    """A tile whose rows and columns one SM of the pair has alone, with many more K steps than stages:
    no wait runs out, and repeated calls give the same bits."""
    x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
    dout = _rows(_gen(M), M, H, torch.bfloat16)
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
    ws = torch.empty(q.qmoe_gated_ffn_backward_workspace_size(M, H, I), dtype=torch.uint8,
                     device="cuda")
    want = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, workspace=ws)
    out = q.qmoe_gated_ffn(x, w13, w2)
    for _ in range(50):
        got = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, workspace=ws)
        assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(out, q.qmoe_gated_ffn(x, w13, w2))
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(113, 520, 328), (129, 72, 2056), (160, 1032, 328), (200, 4096, 96),
                                   (241, 264, 264), (256, 520, 1000), (256, 8, 8)])
def test_gated_ffn_of_large_decode_batches(M, H, I, dtype):
    """The last batches whose tokens are an MMA's columns."""
    ops.test_gated_ffn(M, H, I, "gelu" if M % 2 else "silu", 1.0 if I == 328 else math.inf, dtype)
    if (H, dtype) == (4096, torch.bfloat16):
        ops.test_gated_ffn_odd_tokens_stay_alone(M)


@pytest.mark.parametrize("c", [
    _case(12000, 1001), _case(12000, 1001, torch.float16, gate="full", pad=3),
    _case(30000, 65, gate="channel"), _case(30000, 65, residual=False, post=False),
    _case(30000, 512, torch.float16, residual=False, post=False), _case(3000, 7168),
    _case(12000, 1024, torch.float16, post=False, gate="token"), _case(6000, 1026, torch.float16),
    _case(4000, 2048, torch.float32, residual=False)], ids=lambda c: "-".join(str(v) for v in c.values()))
def test_norms_of_many_rows_a_cta(c):
    """So many rows that each place of a ring of rows is used several times: all rows and sums."""
    ops.test_block_norm(c)
    ops.test_block_norm_backward(c)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gated_ffn_of_the_largest_weights(M):
    """Weights of more than 2^32 elements.  Of w2 only the last 64 columns are other than 0, so that all
    results but h's product are those of these 64 of I, in the last rows of w13's halves."""
    H, I, dt, few = 65536, 32776, torch.bfloat16, 64
    g = _gen(1)
    x, dout = _rows(g, M, H, dt), _rows(g, M, H, dt)
    w13 = torch.empty(2 * I, H, dtype=dt, device="cuda").normal_(0.0, 1.5 * H ** -0.5, generator=g)
    w2 = torch.zeros(H, I, dtype=dt, device="cuda")
    w2[:, -few:].normal_(0.0, few ** -0.5, generator=g)
    s13 = torch.cat([w13[I - few:I], w13[-few:]])
    s2 = w2[:, -few:].contiguous()
    r, u = ROUND[dt], ops.U
    _, _, h, eh = ops._up("silu", math.inf, x, s13)
    eh = eh + r * (h.abs() + eh)
    w = s2.double()
    ref = h @ w.t()
    bound = eh @ w.abs().t() + (few + 4) * 2 * u * ((h.abs() + eh) @ w.abs().t())
    _near(q.qmoe_gated_ffn(x, w13, w2), ref, bound + r * (ref.abs() + bound), "out")
    out, (kept,) = q.qmoe_gated_ffn_saved(x, w13, w2)
    _near(out, ref, bound + r * (ref.abs() + bound), "out beside what is kept")
    dx, dw13, dw2 = q.qmoe_gated_ffn_backward(dout, x, w13, w2, (kept,))
    kept = kept.double()
    for at, where in ((slice(I - few, I), "the last"), (slice(0, few), "the first")):
        half = slice(at.start + I, at.stop + I)
        want = _ffn_grads("silu", math.inf, dout, x, torch.cat([w13[at], w13[half]]), w2[:, at],
                          kept[:, at], kept[:, half], dt)
        if where == "the last":
            _near(dx, *want["dx"], "dx")
        _near(torch.cat([dw13[at], dw13[half]]), *want["dw13"], "dw13, " + where)
        _near(dw2[:, at], *want["dw2"], "dw2, " + where)
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)
