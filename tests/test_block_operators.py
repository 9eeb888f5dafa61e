"""The norms around a block, activation checkpoints in 8 bits and the gated feed-forward block:
refusals (CPU) and parity with plain 64-bit forms (GPU).

Tolerances.  u = 2^-24 is fp32's unit roundoff, r a type's (half its epsilon) and `tiny` half a
step of fp16's subnormals.  A sum of n products in fp32 in any order is within n u sum|terms| of
the exact one; tensor-core additions truncate, which doubles u.  A few more operations on a value
add a few u each: 16 u stands for all of them where nothing is said.  The gated block's
activation goes through approximations of exp and division of a few 2^-22: relative 2^-19.
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
HALVES = DTYPES[:2]
gpu = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, width, dtype, pad=0, offset=0, std=1.0):
    t = (std * torch.randn(n, width + pad + offset, generator=g, device="cuda")).to(dtype)
    return t[:, offset:offset + width]


def _near(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((got - ref).abs().max()),
                           float(torch.as_tensor(bound).max()))


# ================================================================== refusals, no GPU
@pytest.fixture(scope="module")
def lib():
    from quantized_moe_grouped_route_gb300 import build
    build.build()
    return qmoe.lib()


P = ctypes.c_void_p
ARG, SHAPE, WS, OK = (qmoe.QMOE_ERR_ARG, qmoe.QMOE_ERR_SHAPE, qmoe.QMOE_ERR_WORKSPACE,
                      qmoe.QMOE_OK)
A = P(4096)  # never read: what follows is refused before anything is enqueued


def test_norm_refusals(lib):
    def call(dtype=0, y=None, ldy=8, res=None, ldr=8, scale=1.0, gate=None, gdt=0, form=0, ldg=1,
             gating=0, post=None, pre=None, wdt=0, offset=0.0, eps=1e-6, M=4, H=8, out=None,
             normed=None):
        return lib.qmoe_block_norm(y, dtype, ldy, res, ldr, scale, gate, gdt, form, ldg, gating,
                                   post, pre, wdt, offset, eps, M, H, out, normed, None, None, None)
    assert call(dtype=3) == ARG and call(dtype=-1) == ARG
    assert call(scale=math.nan) == ARG and call(offset=math.inf) == ARG
    assert call(eps=-1.0) == ARG and call(eps=math.nan) == ARG and call(eps=math.inf) == ARG
    assert call(H=0) == SHAPE and call(H=65537, ldy=65537) == SHAPE
    assert call(M=-1) == SHAPE and call(M=1 << 27) == SHAPE
    assert call(ldy=7) == SHAPE and call(res=A, ldr=7) == SHAPE
    assert call(gate=A, gdt=1) == ARG and call(gate=A, form=3) == ARG
    assert call(gate=A, gating=2) == ARG and call(gate=P(4097)) == ARG
    assert call(gate=A, ldg=-1) == SHAPE and call(gate=A, form=2, ldg=7) == SHAPE
    assert call(post=A, wdt=1) == ARG and call(pre=P(4098), wdt=2) == ARG
    assert call(pre=A, out=A, y=A) == ARG  # a norm without its output
    assert call(normed=A, y=A) == ARG  # an output without its norm
    assert call() == ARG and call(y=A) == ARG and call(y=P(4097), out=A) == ARG
    assert call(M=0) == OK


def test_norm_backward_refusals(lib):
    n = lib.qmoe_block_norm_backward_workspace_size(4, 8)
    assert n > 256 and lib.qmoe_block_norm_backward_workspace_size(4, 0) == 0
    assert lib.qmoe_block_norm_backward_workspace_size(-1, 8) == 0

    def call(dout=A, ldd=8, dn=None, ldn=8, y=A, dtype=0, out=None, gate=None, form=0, post=None,
             pre=None, prstd=None, rstd=None, M=4, H=8, dy=A, dres=None, dgate=None, dpost=None,
             dpre=None, ws=A, size=n):
        return lib.qmoe_block_norm_backward(dout, ldd, dn, ldn, y, dtype, 8, out, 8, 1.0, gate, 0,
                                            form, 1, 0, post, pre, 0, 0.0, prstd, rstd, M, H, dy,
                                            dres, dgate, dpost, dpre, ws, size, None)
    assert call(dtype=5) == ARG and call(H=0) == SHAPE and call(ldd=7) == SHAPE
    assert call(dn=A, pre=A, rstd=A, ldn=4) == SHAPE
    assert call(dgate=A) == ARG and call(dpost=A) == ARG and call(dpre=A) == ARG
    assert call(dout=None) == ARG and call(y=None) == ARG and call(dy=None) == ARG
    assert call(pre=A, rstd=A) == ARG and call(dn=A) == ARG  # dnormed goes with pre_weight
    assert call(post=A) == ARG and call(pre=A, dn=A) == ARG  # without the norms' scales
    assert call(pre=A, dn=A, rstd=A, post=A, prstd=A) == ARG  # without out
    assert call(pre=A, dn=A, rstd=A, dres=A) == ARG
    assert call(ws=P(4096 + 16)) == ARG and call(size=n - 1) == WS
    assert call(M=0) == OK


def test_checkpoint_refusals(lib):
    def pack(dtype=0, ldx=8, M=4, C=8, x=A, codes=A, scales=A):
        return lib.qmoe_checkpoint8(x, dtype, ldx, M, C, codes, scales, None)

    def restore(dtype=0, M=4, C=8, codes=A, scales=A, out=A):
        return lib.qmoe_checkpoint8_restore(codes, scales, dtype, M, C, out, None)
    for f in (pack, restore):
        assert f(dtype=3) == ARG and f(M=-1) == SHAPE and f(C=0) == SHAPE
        assert f(codes=None) == ARG and f(scales=None) == ARG and f(M=0) == OK
    assert pack(C=(1 << 20) + 1, ldx=1 << 21) == SHAPE
    assert pack(ldx=7) == SHAPE and pack(x=None) == ARG and pack(x=P(4097)) == ARG
    assert restore(out=None) == ARG and restore(out=P(4098), dtype=2) == ARG


def test_ffn_refusals(lib):
    n = lib.qmoe_gated_ffn_workspace_size(4, 64, 128)
    assert n >= 256 + 4 * 128 * 2
    for bad in ((4, 60, 128), (4, 64, 4), (-1, 64, 128), (4, 65544, 8), (1 << 27, 64, 128)):
        assert lib.qmoe_gated_ffn_workspace_size(*bad) == 0
        assert lib.qmoe_gated_ffn_backward_workspace_size(*bad, 16) == 0
    assert lib.qmoe_gated_ffn_backward_workspace_size(4, 64, 128, 4) == 0

    def call(x=A, dtype=0, ldx=64, w13=A, w2=A, act=0, limit=math.inf, M=4, H=64, I=128, out=A,
             kept=None, scales=None, ws=A, size=n):
        return lib.qmoe_gated_ffn(x, dtype, ldx, w13, w2, act, limit, M, H, I, out, kept, scales, ws,
                                  size, None)
    assert call(dtype=2) == ARG and call(act=2) == ARG and call(act=-1) == ARG
    for limit in (0.0, -1.0, math.nan):
        assert call(limit=limit) == ARG and call(limit=limit, M=0) == ARG
    assert call(H=60) == SHAPE and call(I=12) == SHAPE and call(H=0) == SHAPE
    assert call(ldx=63) == SHAPE and call(ldx=68) == SHAPE and call(ldx=0) == SHAPE
    assert call(x=None) == ARG and call(w13=None) == ARG and call(w2=None) == ARG
    assert call(out=None) == ARG and call(ws=None) == ARG and call(scales=A) == ARG
    for k in ("x", "w13", "w2", "out", "kept"):
        assert call(**{k: P(4096 + 8)}) == ARG
    assert call(ws=P(4096 + 64)) == ARG and call(size=n - 1) == WS
    assert call(M=0) == OK

    m = lib.qmoe_gated_ffn_backward_workspace_size(4, 64, 128, 16)
    assert lib.qmoe_gated_ffn_backward_workspace_size(4, 64, 128, 8) > m

    def back(dout=A, dtype=0, ldd=64, x=A, ldx=64, xs=None, w13=A, w2=A, kept=A, ks=None, act=0,
             limit=math.inf, M=4, H=64, I=128, dx=A, dw13=A, dw2=A, ws=A, size=m):
        return lib.qmoe_gated_ffn_backward(dout, dtype, ldd, x, ldx, xs, w13, w2, kept, ks, act,
                                           limit, M, H, I, dx, dw13, dw2, ws, size, None)
    assert back(dtype=2) == ARG and back(act=2) == ARG and back(limit=0.0) == ARG
    assert back(H=60) == SHAPE and back(ldd=68) == SHAPE and back(ldx=56) == SHAPE
    assert back(xs=A) == ARG and back(ks=A) == ARG and back(xs=A, ks=A, ldx=72) == SHAPE
    for k in ("dout", "x", "w13", "w2", "kept", "ws"):
        assert back(**{k: None}) == ARG
    for k in ("dout", "x", "w13", "w2", "kept", "dx", "dw13", "dw2"):
        assert back(**{k: P(4096 + 8)}) == ARG
    assert back(size=m - 1) == WS and back(xs=A, ks=A, size=m) == WS
    assert back(M=0, dw13=None, dw2=None) == OK


# ============================================================================= norms
def _forms(case, s):
    """The definition in 64 bits on the inputs as given: out, normed, and the two scales."""
    v = s["y"].double()
    size = v.abs()  # what v's error is relative to, beside a few u
    H = v.shape[1]
    post = pre = normed = None
    if case["post"]:
        post = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + case["eps"])
        v = v * post * (case["offset"] + s["post"].double())
        size = v.abs() + s["y"].double().abs() * post * abs(case["offset"])
    if s["gate"] is not None:
        g = s["gate"].double()
        g = torch.sigmoid(g) if case["sigmoid"] else g
        v, size = v * g, size * g.abs()
    if s["residual"] is not None:
        r = case["scale"] * s["residual"].double()
        v, size = v + r, size + r.abs()
    if case["pre"]:
        pre = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + case["eps"])
        normed = v * pre * (case["offset"] + s["pre"].double())
    return v, size, normed, post, pre


def _norm_inputs(c, seed):
    g = _gen(seed)
    M, H, dt = c["M"], c["H"], c["dtype"]
    s = {"y": _rows(g, M, H, dt, c["pad"], c["pad"]), "residual": None, "gate": None,
         "post": None, "pre": None}
    if c["residual"]:
        s["residual"] = _rows(g, M, H, dt, c["pad"], std=3.0)
    wdt = torch.float32 if c["fp32"] else dt
    for k in ("post", "pre"):
        if c[k]:
            s[k] = (1.0 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wdt)
    shape = {"token": (M, 1), "channel": (1, H), "full": (M, H)}.get(c["gate"])
    if shape:
        s["gate"] = torch.randn(shape, generator=g, device="cuda").to(wdt)
    return s


def _norm_call(c, s, **kw):
    return q.qmoe_block_norm(s["y"], residual=s["residual"], gate=s["gate"],
                             gating=int(c["sigmoid"]), post_weight=s["post"], pre_weight=s["pre"],
                             residual_scale=c["scale"], weight_offset=c["offset"], eps=c["eps"], **kw)


def _case(M, H, dtype=torch.bfloat16, residual=True, post=True, pre=True, gate=None, sigmoid=False,
          scale=1.0, offset=0.0, pad=0, fp32=False, eps=1e-6):
    return dict(M=M, H=H, dtype=dtype, residual=residual, post=post, pre=pre, gate=gate,
                sigmoid=sigmoid, scale=scale, offset=offset, pad=pad, fp32=fp32, eps=eps)


NORMS = [
    _case(1, 1), _case(1, 8, gate="channel"), _case(3, 7, torch.float16, gate="token"),
    _case(5, 33, torch.float32, gate="full", offset=1.0), _case(2, 256, gate="full", sigmoid=True),
    _case(17, 264, pad=8), _case(17, 264, pad=3, gate="channel", fp32=True),
    _case(9, 1001, torch.float16, gate="channel", scale=0.5), _case(400, 72, gate="token"),
    _case(700, 1024, torch.float32, gate="token", sigmoid=True), _case(330, 4098, pad=2),
    _case(16, 7168), _case(310, 7168, gate="channel", sigmoid=True, scale=-0.25),
    _case(400, 1000, torch.float16, gate="full", fp32=True, pad=8),
    _case(3, 8192, torch.float32, fp32=True), _case(2, 8200, gate="channel", pad=8),
    _case(2, 16385, torch.float16, gate="token"), _case(3, 65536, gate="full"),
    _case(2, 65535, torch.float32, gate="channel", offset=1.0),
    _case(7, 512, post=False), _case(7, 512, pre=False, gate="token"),
    _case(7, 512, residual=False), _case(7, 512, residual=False, post=False),
    _case(340, 2056, torch.float32, residual=False, post=False, offset=1.0),
    _case(7, 512, post=False, pre=False, gate="full", fp32=True, eps=0.0),
]


@gpu
@pytest.mark.parametrize("c", NORMS, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_block_norm(c):
    M, H, dt = c["M"], c["H"], c["dtype"]
    s = _norm_inputs(c, H + M)
    out, normed, post, pre = _norm_call(c, s)
    v, size, n64, post64, pre64 = _forms(c, s)
    changes = c["residual"] or c["post"] or c["gate"] is not None
    # rstd: half the relative error of a sum of H squares, and a few operations
    e = (0.5 * H + 16) * U
    ev = ((e if c["post"] else 0.0) + 16 * U) * size
    if changes:
        _near(out, v, ev + ROUND[dt] * (v.abs() + ev) + TINY[dt], "out")
    else:
        assert out is None
    assert (post is None) == (not c["post"]) and (pre is None) == (not c["pre"])
    if c["post"]:
        _near(post[:, None], post64, e * post64, "post_rstd")
    if c["pre"]:
        # the relative error of the root of a sum of squares: that of the vector under it
        far = ev.norm(dim=1, keepdim=True) / v.norm(dim=1, keepdim=True).clamp(min=1e-300) + e
        _near(pre[:, None], pre64, 1.01 * far * pre64, "pre_rstd")
        w = (c["offset"] + s["pre"].double()).abs() + 2 * U * (s["pre"].double().abs() + c["offset"])
        bound = w * pre64 * (ev + (1.01 * far + 16 * U) * v.abs())
        _near(normed, n64, bound + ROUND[dt] * (n64.abs() + bound) + TINY[dt], "normed")
    for a, b in zip(_norm_call(c, s), (out, normed, post, pre)):
        assert (a is None and b is None) or torch.equal(a, b)
    if changes and c["residual"] and c["pad"] == 0:  # in place of the residual
        into = s["residual"].clone()
        got = _norm_call(c, dict(s, residual=into), out=into)
        assert got[0] is into and torch.equal(into, out)
        assert normed is None or torch.equal(got[1], normed)


def _norm_grads(c, s, out, dout, dn, post, pre):
    """The gradients' formulas in 64 bits on what was kept, with bounds of their errors."""
    H = c["H"]
    y, e = s["y"].double(), (H + 16) * U
    G = torch.zeros_like(y) if dout is None else dout.double()
    eG = 0.0 * G
    r = {}
    if c["pre"]:
        x = (y if out is None else out.double()) * pre.double()[:, None]
        d = dn.double() * (c["offset"] + s["pre"].double())
        ed = 4 * U * dn.double().abs() * (abs(c["offset"]) + s["pre"].double().abs())
        r["dpre"] = ((dn.double() * x).sum(0), (c["M"] + 8) * U * (dn.double() * x).abs().sum(0))
        along, size = (d * x).mean(1, keepdim=True), ((d.abs() + ed) * x.abs()).mean(1, keepdim=True)
        ealong = e * size + (ed * x.abs()).mean(1, keepdim=True)
        p = pre.double()[:, None]
        part = p * (d - x * along)
        eG = 16 * U * (G.abs() + p * (d.abs() + x.abs() * size)) + p * (ed + x.abs() * ealong)
        G = G + part
    if c["residual"]:
        r["dresidual"] = (c["scale"] * G, abs(c["scale"]) * (eG + U * G.abs()))
    a = da = 1.0
    if s["gate"] is not None:
        a = s["gate"].double()
        if c["sigmoid"]:
            a = torch.sigmoid(a)
            da = a * (1.0 - a)
    w = c["offset"] + s["post"].double() if c["post"] else 1.0
    ww = abs(c["offset"]) + s["post"].double().abs() if c["post"] else 1.0
    unit = y * post.double()[:, None] if c["post"] else y
    v, vv = unit * w, unit.abs() * ww
    aa = torch.as_tensor(a).abs()
    if s["gate"] is not None:
        each, eeach = G * v * da, (eG + 16 * U * G.abs()) * vv * da
        if c["gate"] == "full":
            r["dgate"] = (each, eeach)
        else:
            dim = 1 if c["gate"] == "token" else 0
            n = H if c["gate"] == "token" else c["M"]
            r["dgate"] = (each.sum(dim, keepdim=True),
                          (eeach + (n + 16) * U * (G.abs() * vv * da)).sum(dim, keepdim=True))
    dv, edv = G * a, aa * (eG + 16 * U * G.abs())
    if c["post"]:
        r["dpost"] = ((dv * unit).sum(0),
                      ((edv + (c["M"] + 16) * U * dv.abs()) * unit.abs()).sum(0))
        d, dd, ed = dv * w, dv.abs() * ww, edv * ww + 4 * U * dv.abs() * ww
        along, size = (d * unit).mean(1, keepdim=True), (dd * unit.abs()).mean(1, keepdim=True)
        ealong = e * size + (ed * unit.abs()).mean(1, keepdim=True)
        p = post.double()[:, None]
        dv = p * (d - unit * along)
        edv = p * (ed + unit.abs() * ealong) + 16 * U * p * (dd + unit.abs() * size)
    r["dy"] = (dv, edv)
    return r


@gpu
@pytest.mark.parametrize("c", NORMS, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_block_norm_backward(c):
    M, H, dt = c["M"], c["H"], c["dtype"]
    s = _norm_inputs(c, H + M)
    out, normed, post, pre = _norm_call(c, s)
    g = _gen(M)
    dn = _rows(g, M, H, dt, c["pad"]) if c["pre"] else None
    dout = None if out is None else _rows(g, M, H, dt, c["pad"], c["pad"])

    def call(dout, dn, **kw):
        return q.qmoe_block_norm_backward(
            dout, dn, s["y"], out=out, residual=c["residual"], gate=s["gate"],
            gating=int(c["sigmoid"]), post_weight=s["post"], pre_weight=s["pre"], post_rstd=post,
            pre_rstd=pre, residual_scale=c["scale"], weight_offset=c["offset"], **kw)

    got = call(dout, dn)
    want = _norm_grads(c, s, out, dout, dn, post, pre)
    for name, t in zip(("dy", "dresidual", "dgate", "dpost", "dpre"), got):
        assert (t is None) == (name not in want), name
        if t is not None:
            ref, bound = want[name]
            k = t.dtype
            assert k == (dt if name in ("dy", "dresidual") or (name == "dgate" and
                                                              c["gate"] == "full")
                         else torch.float32)
            _near(t, ref, bound + ROUND[k] * (ref.abs() + bound) + TINY[k], name)
    for a, b in zip(call(dout, dn), got):
        assert (a is None and b is None) or torch.equal(a, b)
    if c["pre"] and dout is not None:  # of the norm before the next block alone
        alone = call(None, dn)
        want = _norm_grads(c, s, out, None, dn, post, pre)
        ref, bound = want["dy"]
        _near(alone[0], ref, bound + ROUND[dt] * (ref.abs() + bound) + TINY[dt], "dy of normed")


@gpu
@pytest.mark.parametrize("gate", [None, "token", "channel", "full"])
@pytest.mark.parametrize("M", [1, 0, 37])
def test_block_norm_through_autograd(M, gate):
    """loss.backward() against autograd of the definition in 64 bits, fp32 activations (sums of at
    most H + M = 77 terms: 2^-16 of the largest is far above their rounding), and the loss's slope
    along a direction against a central difference of the definition in 64 bits."""
    H = 40
    c = _case(M, H, torch.float32, gate=gate, sigmoid=True, scale=0.5, offset=1.0)
    s = _norm_inputs(c, 3)
    leaves = {k: t.clone().requires_grad_(True) for k, t in s.items() if t is not None}
    out, normed, *_ = _norm_call(c, {**s, **leaves})
    g = _gen(4)
    a, b = (torch.randn(M, H, generator=g, device="cuda") for _ in range(2))
    ((out * a).sum() + (normed * b).sum()).backward()
    wide = {k: t.double().requires_grad_(True) for k, t in s.items() if t is not None}

    def loss(s64):
        v, _, n, _, _ = _forms(c, {**s, **s64})
        return (v * a.double()).sum() + (n * b.double()).sum()
    loss(wide).backward()
    slope = 0.0
    way = {k: torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
           for k, t in wide.items()}
    for k, t in leaves.items():
        want = wide[k].grad
        if want.numel():
            assert (t.grad.double() - want).abs().max() <= 2.0 ** -16 * want.abs().max()
        assert t.grad.shape == t.shape
        slope += float((t.grad.double() * way[k]).sum())
    with torch.no_grad():
        h = 1e-5
        up, down = (loss({k: t + d * h * way[k] for k, t in wide.items()}) for d in (1, -1))
    # the difference is off by O(h^2), far below the gradients' own rounding
    total = sum(float((t.grad.abs() * way[k].abs()).sum()) for k, t in wide.items())
    assert abs(float(up - down) / (2 * h) - slope) <= 2.0 ** -16 * total + 1e-9


@gpu
def test_block_norm_of_odd_tokens():
    """A token of infinities, NaN or zeros spoils its own row and no other; eps = 0 and a row of
    zeros give NaN there, as the formula does."""
    c = _case(70, 520, gate="token")
    s = _norm_inputs(c, 1)
    good = _norm_call(c, s)
    odd = dict(s, y=s["y"].clone())
    odd["y"][3, 5], odd["y"][40, 0], odd["y"][9] = math.inf, math.nan, 0.0
    got = _norm_call(c, odd)
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[[3, 9, 40]] = False
    for a, b in zip(got, good):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(got[1][[3, 40]]).all() and torch.isfinite(got[1][9]).all()
    assert torch.equal(got[0][9], s["residual"][9])
    zeros = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    _, n, _, pre = q.qmoe_block_norm(zeros, pre_weight=torch.ones(64, device="cuda"), eps=0.0)
    assert torch.isinf(pre).all() and torch.isnan(n).all()


@gpu
def test_block_norm_refuses():
    t = torch.ones
    kw = dict(device="cuda", dtype=torch.bfloat16)
    y, w = t(4, 16, **kw), t(16, **kw)
    for bad in (dict(), dict(residual=t(3, 16, **kw)), dict(residual=t(4, 16, device="cuda")),
                dict(gate=t(4, **kw)), dict(gate=t(3, 1, **kw)), dict(gate=t(4, 2, **kw)),
                dict(gate=t(4, 1, **kw).half()), dict(post_weight=t(15, **kw)),
                dict(post_weight=w, pre_weight=w.float()), dict(pre_weight=w, out=y),
                dict(post_weight=w, normed=y), dict(post_weight=w.cpu()),
                dict(residual=t(16, 4, **kw).t())):
        with pytest.raises(ValueError):
            q.qmoe_block_norm(y, **bad)
    with pytest.raises(qmoe.QmoeError):
        q.qmoe_block_norm(y, post_weight=w, gate=t(4, 1, **kw), gating=2)
    with pytest.raises(ValueError):  # a gradient without its norm
        q.qmoe_block_norm_backward(y, y, y, post_weight=w, post_rstd=t(4, device="cuda"))
    with pytest.raises(ValueError):
        q.qmoe_block_norm(y.requires_grad_(True), post_weight=w, out=torch.empty_like(y))


# ======================================================================= checkpoints
def _ck64(x):
    """The format's definition on the CPU: (codes, scales) of blocks of 32 columns."""
    M, C = x.shape
    B = -(-C // 32)
    p = torch.nn.functional.pad(x.double().cpu(), (0, 32 * B - C)).view(M, B, 32)
    top = p.abs().amax(-1)
    scales = torch.zeros(M, B, dtype=torch.int64)
    for m in range(M):
        for b in range(B):
            v = float(top[m, b])
            if not math.isfinite(v):
                scales[m, b] = 255
                continue
            e = -127
            while v > 127 * 2.0 ** e:
                e += 1
            scales[m, b] = e + 127
    step = torch.exp2(scales.double() - 127)[..., None]
    fine = scales[..., None] < 255
    codes = torch.where(fine, torch.round(torch.where(fine, p / step, 0.0)), 0.0)
    return codes.view(M, -1)[:, :C].to(torch.int8), scales.to(torch.uint8)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C,pad", [(1, 1, 0), (3, 31, 0), (5, 32, 8), (9, 33, 3), (4, 72, 0),
                                     (2, 1000, 8), (7, 2050, 2), (130, 516, 4)])
def test_checkpoint8(M, C, pad, dtype):
    g = _gen(M + C)
    x = _rows(g, M, C, dtype, pad, pad)
    x *= torch.exp2(torch.randint(-12, 4, (M, C), generator=g, device="cuda").float()).to(dtype)
    if M > 2:  # blocks of zeros, of one value, at a border, of the least and largest numbers
        most, least = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
        x[0, :32] = 0.0
        x[1, :16], x[1, 16:32] = 127.0, -126.5
        x[2, :32] = least
        if C > 32:
            x[0, 32:64], x[1, 32:64] = most, 127.5
            x[2, 32:64] = torch.finfo(dtype).smallest_normal / 64
    want = _ck64(x)
    codes, scales = q.qmoe_checkpoint8(x)
    assert torch.equal(scales.cpu(), want[1]) and torch.equal(codes.cpu(), want[0])
    step = torch.exp2(want[1].double() - 127).repeat_interleave(32, 1)[:, :C]
    most = torch.finfo(dtype).max
    value = (want[0].double() * step).clamp(-most, most)
    back = q.qmoe_checkpoint8_restore(codes, scales, dtype)
    assert back.dtype == dtype and torch.equal(back.double().cpu(), value)  # exactly
    assert ((x.double().cpu() - value).abs() <= step / 2).all()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_checkpoint8_of_infinities(dtype):
    x = _rows(_gen(2), 5, 100, dtype)
    good = q.qmoe_checkpoint8_restore(*q.qmoe_checkpoint8(x), dtype)
    x[1, 33], x[3, 99] = math.inf, math.nan
    codes, scales = q.qmoe_checkpoint8(x)
    back = q.qmoe_checkpoint8_restore(codes, scales, dtype)
    assert int(scales[1, 1]) == 255 and int(scales[3, 3]) == 255 and int((scales == 255).sum()) == 2
    for m, cols in ((1, slice(32, 64)), (3, slice(96, 100))):
        assert torch.isnan(back[m, cols]).all()
        back[m, cols] = good[m, cols]
    assert torch.equal(back, good)


@gpu
def test_checkpoint8_refuses():
    x = torch.ones(4, 40, device="cuda", dtype=torch.bfloat16)
    codes, scales = q.qmoe_checkpoint8(x)
    for bad in ((codes, scales[:, :1]), (codes.to(torch.uint8), scales), (codes[:, ::2], scales),
                (codes, scales.cpu())):
        with pytest.raises(ValueError):
            q.qmoe_checkpoint8_restore(*bad)
    with pytest.raises(ValueError):
        q.qmoe_checkpoint8_restore(codes, scales, torch.float64)
    with pytest.raises(ValueError):
        q.qmoe_checkpoint8(x.t())
    with pytest.raises(ValueError):
        q.qmoe_checkpoint8(x, codes=codes[:3])
    assert q.qmoe_checkpoint8(x[:0])[0].shape == (0, 40)


# ============================================================ gated feed-forward block
ACTS = {"silu": 0, "gelu": 1}


def _act(kind, g):
    a = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(
        g, approximate="tanh")
    with torch.enable_grad():
        z = g.detach().clone().requires_grad_(True)
        b = torch.nn.functional.silu(z) if kind == "silu" else torch.nn.functional.gelu(
            z, approximate="tanh")
        d, = torch.autograd.grad(b.sum(), z)
    return a, d


def _ffn_inputs(M, H, I, dtype, pad=0, seed=0):
    g = _gen(seed + M + H + I)
    x = _rows(g, M, H, dtype, pad)
    w13 = _rows(g, 2 * I, H, dtype, std=1.5 * H ** -0.5)
    w2 = _rows(g, H, I, dtype, std=I ** -0.5)
    return x, w13, w2


SLOPE = 1.13  # the largest of either activation's derivatives (SiLU 1.0998, tanh GELU 1.129)


def _up(kind, limit, x, w13):
    """u, g, h in 64 bits and bounds of the kernel's errors in them (h before its rounding)."""
    x, w = x.double(), w13.double()
    I, H = w.shape[0] // 2, w.shape[1]
    ug, size = x @ w.t(), x.abs() @ w.abs().t()
    eug = (H + 4) * 2 * U * size
    u, g, eu, eg = ug[:, :I], ug[:, I:], eug[:, :I], eug[:, I:]
    a, _ = _act(kind, g.clamp(max=limit))
    v = u.clamp(-limit, limit)
    h = a * v
    eh = (a.abs() + SLOPE * eg) * eu + SLOPE * eg * v.abs() + 2.0 ** -19 * h.abs()
    return ug, eug, h, eh


SIZES = [(1, 64, 64), (1, 8, 8), (2, 72, 40), (8, 1024, 264), (9, 256, 1000), (16, 520, 128),
         (33, 2048, 136), (64, 512, 512), (100, 200, 72), (128, 768, 1536), (129, 64, 200),
         (255, 1160, 328), (257, 328, 136), (300, 4096, 96), (513, 264, 520), (1000, 512, 264),
         (2050, 136, 72)]


@gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,H,I", SIZES)
@pytest.mark.parametrize("kind,limit", [("silu", math.inf), ("gelu", 1.0)])
def test_gated_ffn(M, H, I, kind, limit, dtype):
    x, w13, w2 = _ffn_inputs(M, H, I, dtype, pad=8 if M % 2 else 0)
    n = q.qmoe_gated_ffn_workspace_size(M, H, I)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xAB)
    behind = torch.full((M + 3, H), 7.0, dtype=dtype, device="cuda")
    how = dict(activation=ACTS[kind], limit=limit)
    out = q.qmoe_gated_ffn(x, w13, w2, workspace=ws, out=behind[:M], **how)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
    _, _, h, eh = _up(kind, limit, x, w13)
    r, tiny, w = ROUND[dtype], TINY[dtype], w2.double()
    eh = eh + r * (h.abs() + eh) + tiny
    ref = h @ w.t()
    bound = eh @ w.abs().t() + (I + 4) * 2 * U * ((h.abs() + eh) @ w.abs().t())
    _near(out, ref, bound + r * (ref.abs() + bound) + tiny, "out")
    assert (behind[M:] == 7.0).all()
    assert torch.equal(out, q.qmoe_gated_ffn(x, w13, w2, **how))
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)


@gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,H,I", [s for s in SIZES if s[0] in (1, 9, 100, 257, 513, 2050)])
@pytest.mark.parametrize("kind,limit", [("silu", math.inf), ("gelu", 1.0)])
def test_gated_ffn_saved(M, H, I, kind, limit, dtype):
    x, w13, w2 = _ffn_inputs(M, H, I, dtype)
    how = dict(activation=ACTS[kind], limit=limit)
    ug, eug, h, eh = _up(kind, limit, x, w13)
    r, tiny, w = ROUND[dtype], TINY[dtype], w2.double()
    eh = eh + r * (h.abs() + eh) + tiny
    ref = h @ w.t()
    bound = eh @ w.abs().t() + (I + 4) * 2 * U * ((h.abs() + eh) @ w.abs().t())
    bound = bound + r * (ref.abs() + bound) + tiny
    out, (kept,) = q.qmoe_gated_ffn_saved(x, w13, w2, **how)
    _near(out, ref, bound, "out")
    _near(kept, ug, eug + r * (ug.abs() + eug) + tiny, "u beside g")
    out8, (codes, scales, xc, xs) = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=8, **how)
    assert torch.equal(out8, out)
    want = q.qmoe_checkpoint8(x)
    assert torch.equal(xc, want[0]) and torch.equal(xs, want[1])
    B = -(-I // 32)
    for half in range(2):
        s = scales[:, half * B:(half + 1) * B].double()
        at = slice(half * I, (half + 1) * I)
        step = torch.exp2(s - 127).repeat_interleave(32, 1)[:, :I]
        c = codes[:, at].double()
        _near(c * step, ug[:, at], step / 2 + eug[:, at], "u, g in 8 bits")
        # the scale is the least that fits: twice a block's largest code is past 127, but for
        # rounding and the value's error
        top = torch.nn.functional.pad(c.abs(), (0, 32 * B - I)).view(M, B, 32).amax(-1)
        assert (top <= 127).all() and ((top >= 63) | (s == 0)).all()


def _ffn_grads(kind, limit, dout, x, w13, w2, u, g, dtype):
    r, tiny = ROUND[dtype], TINY[dtype]
    M, H, I = x.shape[0], x.shape[1], u.shape[1]
    d, x, w13, w2 = (t.double() for t in (dout, x, w13, w2))
    a, da = _act(kind, g.clamp(max=limit))
    v = u.clamp(-limit, limit)
    hu = torch.where(u.abs() <= limit, a, 0.0)
    hg = torch.where(g <= limit, da * v, 0.0)
    h = a * v
    dh = d @ w2
    edh = (H + 4) * 2 * U * (d.abs() @ w2.abs())
    # the derivative's two terms can cancel: its error is relative to both
    c = g.clamp(max=limit).abs()
    slope = torch.ones_like(c) if kind == "silu" else 1.6 * (1 + 0.135 * c * c)
    p = torch.where(g.clamp(max=limit) == 0, 0.5, a / g.clamp(max=limit))
    terms = torch.where(g <= limit, (p + c * p * (1 - p) * slope) * v.abs(), 0.0)
    rel = 2.0 ** -19
    dug = torch.cat([dh * hu, dh * hg], 1)
    edug = torch.cat([edh * hu.abs() + rel * (dh * hu).abs(), edh * hg.abs() + rel * dh.abs() * terms], 1)
    edug = edug + r * (dug.abs() + edug) + tiny
    eh = rel * h.abs() + r * h.abs() * (1 + rel) + tiny

    def product(a, ea, b, n):
        ref, size = a @ b, (a.abs() + ea) @ b.abs()
        bound = ea @ b.abs() + (n + 4) * 2 * U * size
        return ref, bound + r * (ref.abs() + bound) + tiny
    dw2, edw2 = product(h.t(), eh.t(), d, M)
    return {"dx": product(dug, edug, w13, 2 * I), "dw13": product(dug.t(), edug.t(), x, M),
            "dw2": (dw2.t(), edw2.t())}


@gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,H,I", [s for s in SIZES if s[0] in (1, 2, 9, 100, 128, 257, 513, 2050)])
@pytest.mark.parametrize("kind,limit,bits", [("silu", math.inf, 16), ("gelu", 1.0, 16),
                                             ("silu", 1.0, 8), ("gelu", math.inf, 8)])
def test_gated_ffn_backward(M, H, I, kind, limit, bits, dtype):
    x, w13, w2 = _ffn_inputs(M, H, I, dtype, pad=8 if M % 2 else 0)
    how = dict(activation=ACTS[kind], limit=limit)
    dout = _rows(_gen(M), M, H, dtype, pad=8 if M % 2 else 0)
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits, **how)
    ws = torch.empty(q.qmoe_gated_ffn_backward_workspace_size(M, H, I, bits), dtype=torch.uint8,
                     device="cuda").fill_(0xAB)
    got = q.qmoe_gated_ffn_backward(dout, None if bits == 8 else x, w13, w2, saved, workspace=ws,
                                    **how)
    assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
    if bits == 8:
        B = -(-I // 32)
        u, g = (saved[0][:, i * I:(i + 1) * I].double() *
                torch.exp2(saved[1][:, i * B:(i + 1) * B].double() - 127)
                .repeat_interleave(32, 1)[:, :I] for i in range(2))
        x = q.qmoe_checkpoint8_restore(*saved[2:], dtype)
    else:
        u, g = saved[0][:, :I].double(), saved[0][:, I:].double()
    want = _ffn_grads(kind, limit, dout, x, w13, w2, u, g, dtype)
    for name, t in zip(("dx", "dw13", "dw2"), got):
        assert t.dtype == dtype
        _near(t, *want[name], name)
    again = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, **how)
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)
    for a, b in zip(again, got):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("M", [0, 1, 70])
def test_gated_ffn_through_autograd(M, bits):
    """loss.backward() is the explicit calls; and the explicit gradient's slope along a direction
    is a central difference of the block in 64 bits: of values near 1, M H terms each off by a
    bf16 rounding or two (and an 8-bit step, a 128th of a block's largest)."""
    H, I = 64, 96
    x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
    leaves = [t.clone().requires_grad_(True) for t in (x, w13, w2)]
    out = q.qmoe_gated_ffn(*leaves, checkpoint=bits, limit=2.0)
    dout = _rows(_gen(9), M, H, torch.bfloat16)
    out.backward(dout)
    want, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits, limit=2.0)
    assert torch.equal(out, want)
    grads = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, limit=2.0)
    for t, g in zip(leaves, grads):
        assert torch.equal(t.grad, g) and g.shape == t.shape
    if M == 0:
        assert not grads[1].any() and not grads[2].any()
        return
    # an expanded gradient, and of one leaf alone
    w = w13.clone().requires_grad_(True)
    q.qmoe_gated_ffn(x, w, w2, checkpoint=bits).sum().backward()
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits)
    ones = torch.ones(M, H, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(w.grad, q.qmoe_gated_ffn_backward(ones, x, w13, w2, saved)[1])

    def loss(x, w13, w2):
        ug = x @ w13.t()
        a = torch.nn.functional.silu(ug[:, I:].clamp(max=2.0))
        return (((a * ug[:, :I].clamp(-2.0, 2.0)) @ w2.t()) * dout.double()).sum()
    g = _gen(10)
    wide = [t.double() for t in (x, w13, w2)]
    way = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in wide]
    way[1] *= H ** -0.5
    way[2] *= I ** -0.5
    h = 1e-6
    slope = float(loss(*(t + h * v for t, v in zip(wide, way))) -
                  loss(*(t - h * v for t, v in zip(wide, way)))) / (2 * h)
    got = sum(float((t.double() * v).sum()) for t, v in zip(grads, way))
    # each gradient's relative error is at most a handful of roundings, random in sign: against
    # the norms' product that is far inside
    size = sum(float(t.double().norm() * v.norm()) for t, v in zip(grads, way))
    assert abs(got - slope) <= (2.0 ** -6 if bits == 8 else 2.0 ** -7) * size


@gpu
@pytest.mark.parametrize("M", [1, 5, 20, 100, 300])
def test_gated_ffn_odd_tokens_stay_alone(M):
    H, I = 512, 264
    x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
    good, _ = q.qmoe_gated_ffn_saved(x, w13, w2)
    plain = q.qmoe_gated_ffn(x, w13, w2)
    at = torch.arange(0, M, 3, device="cuda")
    x[at[::2], 5], x[at[1::2], 7] = math.inf, math.nan
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[at] = False
    out, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
    assert torch.equal(out[keep], good[keep]) and torch.isnan(out[at]).all()
    out = q.qmoe_gated_ffn(x, w13, w2)
    assert torch.equal(out[keep], plain[keep]) and torch.isnan(out[at]).all()
    dout = _rows(_gen(1), M, H, torch.bfloat16)
    dx, _, _ = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved)
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[at]).any(1).all()


@gpu
def test_gated_ffn_refuses():
    kw = dict(device="cuda", dtype=torch.bfloat16)
    t = torch.ones
    x, w13, w2 = t(4, 64, **kw), t(48, 64, **kw), t(64, 24, **kw)
    q.qmoe_gated_ffn(x, w13, w2)
    for bad in ((x.float(), w13.float(), w2.float()), (x, w13[:47], w2), (x.half(), w13, w2),
                (x[:, :56], w13, w2), (x, w13.t().contiguous().t(), w2), (x.cpu(), w13, w2),
                (x[0], w13, w2)):
        with pytest.raises(ValueError):
            q.qmoe_gated_ffn(*bad)
    with pytest.raises(ValueError):
        q.qmoe_gated_ffn(x, w13, w2, checkpoint=4)
    with pytest.raises(ValueError):
        q.qmoe_gated_ffn(x, w13, w2, out=t(3, 64, **kw))
    for how in (dict(activation=2), dict(limit=0.0), dict(limit=math.nan)):
        with pytest.raises(qmoe.QmoeError):
            q.qmoe_gated_ffn(x, w13, w2, **how)
    with pytest.raises(qmoe.QmoeError):  # rows off the 16-byte grid
        q.qmoe_gated_ffn(t(4, 68, **kw)[:, :64], w13, w2)
    with pytest.raises(qmoe.QmoeError):
        q.qmoe_gated_ffn(x, w13, w2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q.qmoe_gated_ffn(x.clone().requires_grad_(True), w13, w2, out=torch.empty_like(x))
    _, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
    _, saved8 = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=8)
    for dout, given, kept in ((x[:3], x, saved), (x, None, saved), (x, x, saved8[:3]),
                              (x, x, (saved[0][:, :24],)), (x, x, ()),
                              (x, x, (saved8[0], saved8[1][:, :1], *saved8[2:]))):
        with pytest.raises(ValueError):
            q.qmoe_gated_ffn_backward(dout, given, w13, w2, kept)


# ================================================================== together, as used
def _train_block(x, weights, bits):
    """A block as a model has it: norm, gated block, norm with gate and residual, next norm."""
    n = q.qmoe_block_norm(x, pre_weight=weights["first"])[1]
    y = q.qmoe_gated_ffn(n, weights["w13"], weights["w2"], checkpoint=bits)
    out, n, *_ = q.qmoe_block_norm(y, residual=x, gate=weights["gate"],
                                   gating=q.QMOE_GATING_SIGMOID, post_weight=weights["post"],
                                   pre_weight=weights["next"], residual_scale=0.5)
    return out, n


def _block64(x, w):
    def rms(v):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    ug = (rms(x) * w["first"]) @ w["w13"].t()
    I = w["w2"].shape[1]
    y = (torch.nn.functional.silu(ug[:, I:]) * ug[:, :I]) @ w["w2"].t()
    v = rms(y) * w["post"]
    out = 0.5 * x + torch.sigmoid(w["gate"]) * v
    return out, rms(out) * w["next"], v


def _block_inputs(M, H, I):
    g = _gen(M)
    x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
    vec = {k: 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda") for k in ("first", "post", "next")}
    return x, dict(vec, w13=w13, w2=w2, gate=torch.randn(M, 1, generator=g, device="cuda"))


@gpu
@pytest.mark.parametrize("M", [1, 6, 50, 333])
@pytest.mark.parametrize("bits", [16, 8])
def test_a_block_of_them(M, bits):
    """Outputs and gradients of the chain against the definition in 64 bits.  Each link rounds to
    bf16 (relative 2^-8 at most a value, about 2^-9.8 in the 2-norm); a gradient passes through
    five to eight roundings and, in 8 bits, through checkpoints off by 2^-7.6 / sqrt(3) of a
    block's largest or about 2^-6.5 of its root mean square.  In the 2-norm all of that stays
    within 2^-5 (8 bits: 2^-4), while a missing or doubled term is of the order of 1.

    A token's gate has one gradient, s (1 - s) <G, v> with G that of out and v the normed y, a sum
    over the row whose terms cancel (one of 0.07 where |G| |v| s (1 - s) is 70): errors dG and dv
    of the two move it by <dG, v> + <G, dv>, so by Cauchy and Schwarz by at most their relative
    errors times |G| |v| s (1 - s), which is what it is held to."""
    H, I = 256, 392
    x, w = _block_inputs(M, H, I)
    leaves = {k: t.clone().requires_grad_(True) for k, t in dict(w, x=x).items()}
    out, n = _train_block(leaves["x"], leaves, bits)
    wide = {k: t.double().requires_grad_(True) for k, t in dict(w, x=x).items()}
    out64, n64, v64 = _block64(wide["x"], wide)
    out64.retain_grad()
    g = _gen(8)
    a, b = (torch.randn(M, H, generator=g, device="cuda") for _ in range(2))
    ((out.float() * a).sum() + (n.float() * b).sum()).backward()
    ((out64 * a.double()).sum() + (n64 * b.double()).sum()).backward()
    tol = 2.0 ** -4 if bits == 8 else 2.0 ** -5
    pairs = [(out, out64), (n, n64)] + [(t.grad, wide[k].grad) for k, t in leaves.items()]
    sigma = torch.sigmoid(wide["gate"].detach())
    gate_size = (sigma * (1 - sigma)) * out64.grad.norm(dim=1, keepdim=True) * \
        v64.detach().norm(dim=1, keepdim=True)
    for got, want in pairs:
        assert got.shape == want.shape
        size = gate_size if want is wide["gate"].grad else want
        assert (got.double() - want).norm() <= tol * size.norm()


@gpu
def test_streams_and_graphs():
    cases = {M: _block_inputs(M, 256, 392) for M in (1, 40, 300)}

    def chain(x, w, stream=None):
        r = []
        for M, (x, w) in cases.items():
            how = dict(post_weight=w["post"], pre_weight=w["next"], gate=w["gate"])
            n = q.qmoe_block_norm(x, pre_weight=w["first"], stream=stream)[1]
            y, saved = q.qmoe_gated_ffn_saved(n, w["w13"], w["w2"], checkpoint=8, stream=stream)
            z = q.qmoe_gated_ffn(n, w["w13"], w["w2"], stream=stream)
            out, n2, p1, p2 = q.qmoe_block_norm(y, residual=x, stream=stream, **how)
            dy, *more = q.qmoe_block_norm_backward(x, n, y, out=out, post_rstd=p1, pre_rstd=p2,
                                                   stream=stream, **how)
            grads = q.qmoe_gated_ffn_backward(dy, None, w["w13"], w["w2"], saved, stream=stream)
            back = q.qmoe_checkpoint8_restore(*saved[2:], stream=stream)
            r += [n, y, z, out, n2, p1, p2, dy, *more, *grads, back, *saved]
        return r
    want = chain(*cases[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        got = chain(*cases[1], stream=given)
        side.synchronize()
        for u, v in zip(want, got):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(*cases[1])
    for x, w in cases.values():
        x.mul_(0.5)
        w["w2"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(chain(*cases[1]), got):
        assert torch.equal(u, v)


@gpu
def test_a_captured_training_step():
    """Forward and backward captured whole (no eager graph of the leaves alive), replayed on new
    inputs."""
    x, w = _block_inputs(70, 256, 392)
    leaves = {k: t.clone().requires_grad_(True) for k, t in dict(w, x=x).items()}
    names = sorted(leaves)

    def step():
        out, n = _train_block(leaves["x"], leaves, 8)
        return torch.autograd.grad((out.float().sum() + n.float().square().sum()),
                                   [leaves[k] for k in names])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        leaves["x"].mul_(-0.5)
        leaves["post"].add_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(step(), got):
        assert torch.equal(a, b)
