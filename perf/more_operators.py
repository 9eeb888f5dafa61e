"""Cases of the dense side of a block: the norms around it fused with its gate and residual, the
gated feed-forward block (a shared expert, or a dense layer's), and activation checkpoints in
8 bits with their use in that block's backward pass.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded once at the
end) and the call a user makes of the library (`own`).
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_BLOCK = 32  # columns that share a checkpoint's scale


def listed():
    return [
        # one request's next token through a shared expert: the weights' stream
        _ffn("ffn_decode_m1_h7168_i2048", 1, 7168, 2048),
        # a decode batch of many requests
        _ffn("ffn_decode_m48_h4096_i1536", 48, 4096, 1536, dtype="fp16"),
        # a ragged prefill batch through a tanh-GELU block with the layer's clamp
        _ffn("ffn_prefill_m2047_h4096_i1536", 2047, 4096, 1536, dtype="fp16", activation="gelu",
             limit=2.0),
        # a large prefill batch
        _ffn("ffn_prefill_m8192_h7168_i2048", 8192, 7168, 2048),
        # its gradients in training, from the pre-activations that the forward pass kept
        _ffn("ffn_backward_m8192_h7168_i2048", 8192, 7168, 2048, mode="backward"),
        # a ragged batch's gradients from activations kept in 8 bits
        _ffn("ffn_backward8_m1023_h4096_i1000", 1023, 4096, 1000, mode="backward", checkpoint=8),
        # a whole training step that keeps its activations in 8 bits between the passes
        _ffn("ffn_step8_m4096_h4096_i1536", 4096, 4096, 1536, mode="step", checkpoint=8),
        # a layer's activations to 8 bits and back
        _checkpoint("checkpoint8_m8192_c7168", 8192, 7168),
        # between two blocks of one decode step: launch latency
        _norm("norm_decode_m16_h7168", 16, 7168),
        # between two blocks of a large prefill batch: bandwidth
        _norm("norm_prefill_m8192_h7168", 8192, 7168, gate="token", sigmoid=True),
        # its gradients
        _norm("norm_backward_m8192_h7168", 8192, 7168, direction="backward"),
        # a learned gate per channel, an odd width that no vector divides
        _norm("norm_backward_m1023_h1001", 1023, 1001, dtype="fp16", gate="channel", scale=0.5,
              direction="backward"),
    ]


def _ffn(name, M, H, I, dtype="bf16", activation="silu", limit=0.0, mode="forward", checkpoint=16,
         pad=0):
    """limit 0: none; checkpoint: bits of the activations kept for the backward pass."""
    return {"name": name, "op": "ffn", "M": M, "H": H, "I": I, "dtype": dtype,
            "activation": activation, "limit": limit, "mode": mode, "checkpoint": checkpoint,
            "pad": pad}


def _checkpoint(name, M, C, dtype="bf16", pad=0):
    return {"name": name, "op": "checkpoint", "M": M, "C": C, "dtype": dtype, "pad": pad}


def _norm(name, M, H, dtype="bf16", residual=True, post=True, pre=True, gate="none", sigmoid=False,
          scale=1.0, offset=0.0, pad=0, direction="forward"):
    """residual, post, pre: which of the residual and the two norms there are."""
    return {"name": name, "op": "norm", "M": M, "H": H, "dtype": dtype, "residual": residual,
            "post": post, "pre": pre, "gate": gate, "sigmoid": sigmoid, "scale": scale,
            "offset": offset, "pad": pad, "direction": direction}


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ffn", "ffn", "ffn", "ffn", "checkpoint", "norm", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "ffn":
        mode = rng.choice(["forward", "forward", "backward", "step"])
        H, I = 8 * spread(8, 1024), 8 * spread(8, 512)
        passes = {"forward": 1, "backward": 2, "step": 3}[mode]
        M = min(spread(1, 8192), max(1, 2 * 8192 * 7168 * 2048 // (H * I * passes)))
        c = _ffn("", M, H, I, dtype=dtype, activation=rng.choice(["silu", "silu", "gelu"]),
                 limit=rng.choice([0.0, 0.0, 2.0]), mode=mode,
                 checkpoint=8 if mode == "step" else rng.choice([8, 16]), pad=rng.choice([0, 0, 8]))
        return {k: v for k, v in c.items() if k != "name"}
    H = spread(64, 8192)
    if rng.random() < 0.6:
        H = (H + 7) // 8 * 8
    dtype = rng.choice([dtype, dtype, "fp32"])
    M = min(spread(1, 16384), max(1, 8192 * 7168 * 2 // (H * _SIZE[dtype])))
    if op == "checkpoint":
        c = _checkpoint("", M, H, dtype=dtype, pad=rng.choice([0, 0, 8, 3]))
    else:
        first = rng.random() < 0.2  # the norm before a model's first block: nothing to add to
        forms = ["none", "token", "channel"] + ["full"] * (M > 1)
        c = _norm("", M, H, dtype=dtype, residual=not first, post=not first and rng.random() < 0.7,
                  pre=first or rng.random() < 0.8,
                  gate="none" if first else rng.choice(forms),
                  sigmoid=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 0.5]),
                  offset=rng.choice([0.0, 1.0]), pad=rng.choice([0, 0, 8, 3]),
                  direction=rng.choice(["forward", "backward"]))
    del c["name"]
    return c


def work(case):
    c = case
    M, es = c["M"], _SIZE[c["dtype"]]
    if c["op"] == "checkpoint":
        blocks = -(-c["C"] // _BLOCK)
        return {"bytes": M * (2 * c["C"] * es + 2 * c["C"] + 2 * blocks), "flops": 4 * M * c["C"]}
    H = c["H"]
    if c["op"] == "ffn":
        I = c["I"]
        weights, rows = 3 * H * I * es, M * H * es
        kept = M * 2 * I * es
        if c["checkpoint"] == 8:
            kept = M * (2 * I + 2 * -(-I // _BLOCK))
        if c["mode"] == "forward":
            return {"bytes": weights + 2 * rows, "flops": 6 * M * H * I}
        if c["mode"] == "backward":  # dout, x, what was kept -> dx, and the weights' gradients
            x = M * (H + -(-H // _BLOCK)) if c["checkpoint"] == 8 else rows
            return {"bytes": 2 * weights + 2 * rows + x + kept, "flops": 12 * M * H * I}
        return {"bytes": 2 * weights + 4 * rows, "flops": 18 * M * H * I}
    vectors = 4 * H * (c["post"] + c["pre"])
    full, plain = c["gate"] == "full", not c["post"] and c["gate"] == "none"
    first = plain and not c["residual"]  # out is y itself
    if c["direction"] == "forward":  # y, residual, gate -> out, normed
        mats = 1 + c["residual"] + full + (not first) + c["pre"]
    else:  # y or none of it, dout, out, dnormed, gate -> dy, dresidual, dgate
        mats = (first or not plain) + (not first) * (1 + c["pre"]) + c["pre"] + full
        mats += 1 + c["residual"] + full
        vectors *= 2
    return {"bytes": M * H * es * mats + vectors, "flops": 10 * M * H}


# ------------------------------------------------------------------------- inputs
def _rows(g, n, width, dtype, pad=0, std=1.0):
    """[n][width] values ~ N(0, std), rows `pad` elements further apart than their width."""
    t = torch.empty(n, width + pad, dtype=dtype, device="cuda")
    t.normal_(0.0, std, generator=g)
    return t[:, :width]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, dt, pad = c["M"], _DT[c["dtype"]], c["pad"]
    s = {"case": c}
    if c["op"] == "checkpoint":
        # activations: a few channels are much larger than the others
        x = torch.empty(M, c["C"] + pad, dtype=torch.float32, device="cuda")
        x.normal_(0.0, 1.0, generator=g)
        x *= torch.exp(torch.randn(c["C"] + pad, generator=g, device="cuda"))
        s["x"] = x.to(dt)[:, :c["C"]]
    elif c["op"] == "ffn":
        H, I = c["H"], c["I"]
        s["x"] = _rows(g, M, H, dt, pad)
        s["w13"] = _rows(g, 2 * I, H, dt, 0, H ** -0.5)
        s["w2"] = _rows(g, H, I, dt, 0, I ** -0.5)
        if c["mode"] != "forward":
            s["dout"] = _rows(g, M, H, dt, pad)
        if c["mode"] == "backward":
            ug = s["x"].float() @ s["w13"].float().t()
            if c["checkpoint"] == 8:
                s["saved"] = _halves_to_8(ug) + _to_8(s.pop("x").float())
            else:
                s["saved"] = (ug.to(dt),)
    else:
        H = c["H"]
        s["y"] = _rows(g, M, H, dt, pad, 0.5)
        s["residual"] = _rows(g, M, H, dt, pad, 3.0) if c["residual"] else None
        for which in ("post", "pre"):
            w = 1.0 - c["offset"] + 0.2 * torch.randn(H, generator=g, device="cuda")
            s[which] = w.to(dt) if c[which] else None
        shape = {"none": None, "token": (M, 1), "channel": (1, H), "full": (M, H)}[c["gate"]]
        s["gate"] = None
        if shape:
            s["gate"] = torch.randn(shape, generator=g, device="cuda").to(dt)
        if c["direction"] == "backward":
            s["saved"] = tuple(_norm_forward(c, s))
            s["dnormed"] = _rows(g, M, H, dt, pad) if c["pre"] else None
            s["dout"] = _rows(g, M, H, dt, pad) if s["saved"][0] is not None else None
    return s


# -------------------------------------------------------------- checkpoints in 8 bits
def _to_8(x):
    """(codes int8 [M][C], scales uint8 [M][blocks]): x = code * 2^(scale - 127), the least
    power of two for which a block's codes are within 127; 255 for a block that is not finite."""
    M, C = x.shape
    blocks = -(-C // _BLOCK)
    p = torch.nn.functional.pad(x, (0, blocks * _BLOCK - C)).view(M, blocks, _BLOCK)
    top = p.abs().amax(-1)
    fine = top < math.inf
    part, e = torch.frexp(torch.where(fine, top, 0.0))
    e = e.int() - 7 + (part > 127 / 128).int()
    e = torch.where(top > 0, e, -127).clamp(min=-127)
    codes = torch.round(p * _two_to(-e)[..., None])
    codes = torch.where(fine[..., None], codes, 0.0).to(torch.int8).view(M, -1)[:, :C]
    return codes.contiguous(), torch.where(fine, e + 127, 255).to(torch.uint8)


def _two_to(e):
    """2^e in 32 bits for -127 <= e <= 127."""
    bits = torch.where(e > -127, (e + 127) << 23, 1 << 22)
    return bits.to(torch.int32).view(torch.float32)


def _from_8(codes, scales, dtype):
    """The values that codes and scales stand for, in 32 bits, within dtype's finite range."""
    s = scales.int()
    f = torch.where(s == 255, math.nan, _two_to(s - 127))
    M, C = codes.shape
    f = f[:, :, None].expand(-1, -1, _BLOCK).reshape(M, -1)[:, :C]
    most = torch.finfo(dtype).max
    return torch.clamp(codes.float() * f, -most, most)


def _halves_to_8(ug):
    """Both halves' codes beside each other, and their scales."""
    I = ug.shape[1] // 2
    u, g = _to_8(ug[:, :I]), _to_8(ug[:, I:])
    return torch.cat([u[0], g[0]], 1), torch.cat([u[1], g[1]], 1)


def _halves_from_8(codes, scales, dtype):
    I, B = codes.shape[1] // 2, scales.shape[1] // 2
    return (_from_8(codes[:, :I], scales[:, :B], dtype), _from_8(codes[:, I:], scales[:, B:], dtype))


# -------------------------------------------------------------------- plain forms
def _act(c, g):
    """The activation and its derivative."""
    if c["activation"] == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * g * g))


def _gated(c, u, g):
    """(h, dh/du, dh/dg) of the clamped gate and up."""
    if c["limit"] == 0.0:
        a, da = _act(c, g)
        return a * u, a, da * u
    L = c["limit"]
    a, da = _act(c, torch.clamp(g, max=L))
    v = torch.clamp(u, -L, L)
    return a * v, torch.where(u.abs() <= L, a, 0.0), torch.where(g <= L, da * v, 0.0)


def _ffn_backward(c, dout, x, w13, w2, u, g):
    h, hu, hg = _gated(c, u, g)
    dh = dout @ w2
    dug = torch.cat([dh * hu, dh * hg], 1)
    return {"dx": dug @ w13, "dw13": dug.t() @ x, "dw2": dout.t() @ h}


def _ffn_plain(s):
    c, dt, I = s["case"], _DT[s["case"]["dtype"]], s["case"]["I"]
    w13, w2 = s["w13"].float(), s["w2"].float()
    if c["mode"] == "backward":
        if c["checkpoint"] == 8:
            u, g = _halves_from_8(*s["saved"][:2], dt)
            x = _from_8(*s["saved"][2:], dt)
        else:
            ug, x = s["saved"][0].float(), s["x"].float()
            u, g = ug[:, :I], ug[:, I:]
        out = _ffn_backward(c, s["dout"].float(), x, w13, w2, u, g)
        return {k: v.to(dt) for k, v in out.items()}
    x = s["x"].float()
    ug = x @ w13.t()
    out = {"out": _gated(c, ug[:, :I], ug[:, I:])[0] @ w2.t()}
    if c["mode"] == "step":
        u, g = _halves_from_8(*_halves_to_8(ug), dt)
        out.update(_ffn_backward(c, s["dout"].float(), _from_8(*_to_8(x), dt), w13, w2, u, g))
    return {k: v.to(dt) for k, v in out.items()}


def _checkpoint_plain(s):
    dt = _DT[s["case"]["dtype"]]
    return {"restored": _from_8(*_to_8(s["x"].float()), dt).to(dt)}


_EPS = 1e-6


def _gate_of(c, s):
    """The gate and its derivative in what is given, 1 and 0 without one."""
    if s["gate"] is None:
        return 1.0, 0.0
    a = s["gate"].float()
    if not c["sigmoid"]:
        return a, 1.0
    p = 1.0 / (1.0 + torch.exp(-a))
    return p, p * (1.0 - p)


def _norm_forward(c, s):
    """(out, normed, post_rstd, pre_rstd), None for what the case has not."""
    dt = _DT[c["dtype"]]
    v = s["y"].float()
    post = pre = normed = None
    if c["post"]:
        post = torch.rsqrt(v.square().mean(1) + _EPS)
        v = v * post[:, None] * (c["offset"] + s["post"].float())
    v = v * _gate_of(c, s)[0]
    if c["residual"]:
        v = c["scale"] * s["residual"].float() + v
    if c["pre"]:
        pre = torch.rsqrt(v.square().mean(1) + _EPS)
        normed = (v * pre[:, None] * (c["offset"] + s["pre"].float())).to(dt)
    changed = c["residual"] or c["post"] or c["gate"] != "none"
    return v.to(dt) if changed else None, normed, post, pre


def _norm_plain(s):
    c, dt = s["case"], _DT[s["case"]["dtype"]]
    if c["direction"] == "forward":
        out, normed, post, pre = _norm_forward(c, s)
        return {"out": out, "normed": normed, "post_rstd": post, "pre_rstd": pre}
    out, _, post, pre = s["saved"]
    y = s["y"].float()
    grads = {}
    G = 0.0 if s["dout"] is None else s["dout"].float()
    if c["pre"]:
        unit = (y if out is None else out.float()) * pre[:, None]
        dn = s["dnormed"].float()
        grads["dpre_weight"] = (dn * unit).sum(0)
        d = dn * (c["offset"] + s["pre"].float())
        G = G + pre[:, None] * (d - unit * (d * unit).mean(1, keepdim=True))
    if c["residual"]:
        grads["dresidual"] = (c["scale"] * G).to(dt)
    a, da = _gate_of(c, s)
    v = unit = y
    if c["post"]:
        unit = y * post[:, None]
        v = unit * (c["offset"] + s["post"].float())
    if s["gate"] is not None:
        dgate = G * v * da
        if c["gate"] == "full":
            grads["dgate"] = dgate.to(dt)
        else:
            grads["dgate"] = dgate.sum(1 if c["gate"] == "token" else 0, keepdim=True)
    dy = G * a
    if c["post"]:
        grads["dpost_weight"] = (dy * unit).sum(0)
        d = dy * (c["offset"] + s["post"].float())
        dy = post[:, None] * (d - unit * (d * unit).mean(1, keepdim=True))
    grads["dy"] = dy.to(dt)
    return grads


# --------------------------------------------------------------- the library's calls
def _ffn_own(s):
    import quantized_moe_grouped_route_gb300 as q
    c = s["case"]
    how = {"activation": q.QMOE_ACT_GELU if c["activation"] == "gelu" else q.QMOE_ACT_SILU,
           "limit": c["limit"] or math.inf}
    if c["mode"] == "forward":
        return {"out": q.qmoe_gated_ffn(s["x"], s["w13"], s["w2"], **how)}
    out = {}
    if c["mode"] == "step":
        out["out"], saved = q.qmoe_gated_ffn_saved(s["x"], s["w13"], s["w2"], checkpoint=8, **how)
        x = None
    else:
        saved, x = s["saved"], s.get("x")
    dx, dw13, dw2 = q.qmoe_gated_ffn_backward(s["dout"], x, s["w13"], s["w2"], saved, **how)
    out.update(dx=dx, dw13=dw13, dw2=dw2)
    return out


def _checkpoint_own(s):
    import quantized_moe_grouped_route_gb300 as q
    codes, scales = q.qmoe_checkpoint8(s["x"])
    return {"restored": q.qmoe_checkpoint8_restore(codes, scales, s["x"].dtype)}


def _norm_own(s):
    import quantized_moe_grouped_route_gb300 as q
    c = s["case"]
    how = {"gate": s["gate"], "gating": q.QMOE_GATING_SIGMOID if c["sigmoid"] else
           q.QMOE_GATING_LINEAR, "post_weight": s["post"], "pre_weight": s["pre"],
           "residual_scale": c["scale"], "weight_offset": c["offset"]}
    if c["direction"] == "forward":
        out, normed, post, pre = q.qmoe_block_norm(s["y"], residual=s["residual"], eps=_EPS, **how)
        return {"out": out, "normed": normed, "post_rstd": post, "pre_rstd": pre}
    out, _, post, pre = s["saved"]
    dy, dresidual, dgate, dpost, dpre = q.qmoe_block_norm_backward(
        s["dout"], s["dnormed"], s["y"], out=out, post_rstd=post, pre_rstd=pre,
        residual=c["residual"], **how)
    grads = {"dpre_weight": dpre, "dresidual": dresidual, "dgate": dgate, "dpost_weight": dpost,
             "dy": dy}
    return {k: v for k, v in grads.items() if v is not None}


_PLAIN = {"ffn": _ffn_plain, "checkpoint": _checkpoint_plain, "norm": _norm_plain}
_OWN = {"ffn": _ffn_own, "checkpoint": _checkpoint_own, "norm": _norm_own}


def run(state):
    out = (_OWN if own else _PLAIN)[state["case"]["op"]](state)
    return {k: out[k] for k in sorted(out) if out[k] is not None}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits: gradients by differentiating the
    definition, checkpoints by rounding to a block's step."""
    s = prepare(case, seed)
    out = {"ffn": _exact_ffn, "checkpoint": _exact_checkpoint, "norm": _exact_norm}[case["op"]](case, s)
    return {k: out[k] for k in sorted(out) if out[k] is not None}


def _steps(x):
    """Each element rounded to its block's step, for finite blocks in 64 bits."""
    held = torch.zeros_like(x)
    for k in range(0, x.shape[1], _BLOCK):
        top = x[:, k:k + _BLOCK].abs().amax(1, keepdim=True)
        step = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 127.0)).clamp(min=-127))
        held[:, k:k + _BLOCK] = torch.round(x[:, k:k + _BLOCK] / step) * step
    return held


def _exact_checkpoint(c, s):
    x = s["x"].double()
    most = torch.finfo(s["x"].dtype).max
    return {"restored": _steps(x).clamp(-most, most)}


def _codes_value(codes, scales):
    at = torch.arange(codes.shape[1], device=codes.device) // _BLOCK
    return codes.double() * torch.exp2(scales.double() - 127.0)[:, at]


def _exact_ffn(c, s):
    H, I = c["H"], c["I"]

    def block(u, g, w2):
        if c["limit"]:
            g, u = torch.clamp(g, max=c["limit"]), torch.clamp(u, -c["limit"], c["limit"])
        kind = torch.nn.functional
        a = kind.silu(g) if c["activation"] == "silu" else kind.gelu(g, approximate="tanh")
        return (a * u) @ w2.t()

    w13, w2 = s["w13"].double(), s["w2"].double()
    result = {}
    if c["mode"] == "backward" and c["checkpoint"] == 8:
        codes, scales, xc, xs = s["saved"]
        B = scales.shape[1] // 2
        up, gate = _codes_value(codes[:, :I], scales[:, :B]), _codes_value(codes[:, I:], scales[:, B:])
        x = _codes_value(xc, xs)
    elif c["mode"] == "backward":
        x, ug = s["x"].double(), s["saved"][0].double()
        up, gate = ug[:, :I], ug[:, I:]
    else:
        x = s["x"].double()
        up, gate = x @ w13[:I].t(), x @ w13[I:].t()
        result["out"] = block(up, gate, w2)
        if c["mode"] == "forward":
            return result
        x, up, gate = _steps(x), _steps(up), _steps(gate)
    up, gate, w2 = (t.detach().clone().requires_grad_(True) for t in (up, gate, w2))
    with torch.enable_grad():
        out = block(up, gate, w2)
        du, dg, dw2 = torch.autograd.grad(out, (up, gate, w2), s["dout"].double())
    result["dx"] = du @ w13[:I] + dg @ w13[I:]
    result["dw13"] = torch.cat([du.t() @ x, dg.t() @ x])
    result["dw2"] = dw2
    return result


def _exact_norm(c, s):
    y = s["y"].double()
    d = {k: s[k].double() if s[k] is not None else None for k in ("residual", "post", "pre", "gate")}
    gate = 1.0 if d["gate"] is None else torch.sigmoid(d["gate"]) if c["sigmoid"] else d["gate"]

    def rms(t):
        return torch.sqrt((t * t).sum(1) / c["H"] + _EPS)

    if c["direction"] == "forward":
        z, result = y, {}
        if c["post"]:
            result["post_rstd"] = 1.0 / rms(z)
            z = z / rms(z)[:, None] * (d["post"] + c["offset"])
        z = gate * z
        if c["residual"]:
            z = z + c["scale"] * d["residual"]
        if c["residual"] or c["post"] or d["gate"] is not None:
            result["out"] = z
        if c["pre"]:
            result["pre_rstd"] = 1.0 / rms(z)
            result["normed"] = z / rms(z)[:, None] * (d["pre"] + c["offset"])
        return result
    # what was kept stands for the norms' inputs and scales: a norm's derivative is the scaled
    # projection that leaves the kept direction out
    out, _, post, pre = s["saved"]

    def through(grad, direction, rstd):
        r = rstd.double()[:, None]
        along = torch.einsum("mh,mh->m", grad, direction * r)[:, None] / c["H"]
        return r * (grad - along * direction * r)

    result = {}
    total = torch.zeros_like(y) if s["dout"] is None else s["dout"].double()
    if c["pre"]:
        at = y if out is None else out.double()
        dn = s["dnormed"].double()
        total = total + through(dn * (d["pre"] + c["offset"]), at, pre)
        result["dpre_weight"] = torch.einsum("mh,mh,m->h", dn, at, pre.double())
    if c["residual"]:
        result["dresidual"] = c["scale"] * total
    z = y
    if c["post"]:
        z = y * post.double()[:, None] * (d["post"] + c["offset"])
    if d["gate"] is not None:
        dgate = total * z * (gate - gate * gate if c["sigmoid"] else 1.0)
        axis = {"full": (), "token": (1,), "channel": (0,)}[c["gate"]]
        result["dgate"] = dgate.sum(axis, keepdim=True) if axis else dgate
    dz = total * gate
    if c["post"]:
        result["dpost_weight"] = torch.einsum("mh,mh,m->h", dz, y, post.double())
        dz = through(dz * (d["post"] + c["offset"]), y, post)
    result["dy"] = dz
    return result
