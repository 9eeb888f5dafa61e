"""Cases of the operators around the MoE layer: the expert gate, the tokens sorted by
expert and back, and a shared projection with low-rank adapters of many requests.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded
once at the end) and the call a user makes of the library (`own`).
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # the router of one decode step: sigmoid scores, a selection bias, experts in groups
        _gate("gate_decode_m16_e256_k8", 16, 256, 8, scoring="sigmoid", n_group=8, topk_group=4,
              scale=2.5),
        # the same router over a large prefill batch
        _gate("gate_prefill_m8192_e256_k8", 8192, 256, 8, scoring="sigmoid", n_group=8,
              topk_group=4, scale=2.5),
        # the router's gradient in a training step, softmax over the chosen experts
        _gate("gate_backward_m8192_e128_k8", 8192, 128, 8, direction="backward"),
        # one decode step's tokens in expert order: launch latency
        _sort("sort_decode_m16_h7168_e256_k8", 16, 7168, 256, 8),
        # a large prefill batch in expert order: the copy's bandwidth
        _sort("sort_prefill_m8192_h7168_e256_k8", 8192, 7168, 256, 8),
        # the sort's gradient under skewed routing, with pairs dropped by their capacity
        _sort("sort_backward_m2048_h4096_e128_k8", 2048, 4096, 128, 8, direction="backward",
              routing="zipf", dropped=True),
        # expert outputs back in token order, an odd width that no vector divides
        _unsort("unsort_m1023_h1001_e60_k4", 1023, 1001, 60, 4, dtype="fp16", routing="zipf"),
        # gradients of expert outputs and routing weights in a large training step
        _unsort("unsort_backward_m8192_h7168_e256_k8", 8192, 7168, 256, 8, direction="backward"),
        # a single token of one request through its adapter
        _lora("lora_decode_m1_k7168_n2048_r16", 1, 7168, 2048, 16, 32),
        # a decode batch, a request (and an adapter) a token
        _lora("lora_decode_m48_k2048_n7168_r32", 48, 2048, 7168, 32, 64),
        # a ragged prefill batch of several requests
        _lora("lora_prefill_m2047_k4096_n4096_r16", 2047, 4096, 4096, 16, 16, tokens="requests",
              dtype="fp16"),
        # a large prefill batch
        _lora("lora_prefill_m8192_k7168_n2048_r64", 8192, 7168, 2048, 64, 8, tokens="requests"),
    ]


def _gate(name, M, E, top_k, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
          scale=1.0, dtype="fp32", masked=False, direction="forward"):
    return {"name": name, "op": "gate", "M": M, "E": E, "top_k": top_k, "scoring": scoring,
            "n_group": n_group, "topk_group": topk_group, "renormalize": renormalize,
            "scale": scale, "dtype": dtype, "masked": masked, "direction": direction}


def _sort(name, M, H, E, top_k, dtype="bf16", routing="even", dropped=False, pad=0,
          direction="forward", op="sort"):
    return {"name": name, "op": op, "M": M, "H": H, "E": E, "top_k": top_k, "dtype": dtype,
            "routing": routing, "dropped": dropped, "pad": pad, "direction": direction}


def _unsort(*args, **kw):
    return _sort(*args, op="unsort", **kw)


def _lora(name, M, K, N, R, L, dtype="bf16", tokens="mixed"):
    return {"name": name, "op": "lora", "M": M, "K": K, "N": N, "R": R, "L": L, "dtype": dtype,
            "tokens": tokens}


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gate", "gate", "sort", "unsort", "lora", "lora"])
    if op == "gate":
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * spread(2, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        top_k = rng.randint(1, max(1, min(16, E * topk_group // n_group)))
        c = _gate("", spread(1, 16384), E, top_k, scoring=rng.choice(["softmax", "sigmoid"]),
                  n_group=n_group, topk_group=topk_group, renormalize=rng.random() < 0.7,
                  scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                  masked=rng.random() < 0.3, direction=rng.choice(["forward", "backward"]))
    elif op == "lora":
        most = 8192 * 7168 * 2048
        K = 8 * spread(8, 1024)
        N = spread(64, 8192)
        M = min(spread(1, 8192), max(1, most // (K * N)))
        c = _lora("", M, K, N, 8 * spread(1, 16), spread(1, 64),
                  dtype=rng.choice(["bf16", "bf16", "fp16"]),
                  tokens=rng.choice(["mixed", "requests"]) if M <= 256 else "requests")
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        top_k = rng.randint(1, 12)
        E = spread(top_k, 512)
        H = spread(64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        most = 8192 * 8 * 7168 * 2
        M = min(spread(1, 16384), max(1, most // (top_k * H * _SIZE[dtype])))
        c = _sort("", M, H, E, top_k, dtype=dtype, routing=rng.choice(["even", "zipf"]),
                  dropped=rng.random() < 0.3, pad=rng.choice([0, 0, 8, 3]),
                  direction=rng.choice(["forward", "backward"]), op=op)
    del c["name"]
    return c


def work(case):
    c = case
    es = _SIZE[c["dtype"]]
    M = c["M"]
    if c["op"] == "gate":
        E, k = c["E"], c["top_k"]
        if c["direction"] == "forward":
            return {"bytes": M * E * es + M * k * 8, "flops": 4 * M * E}
        read = M * E * es if c["scoring"] == "softmax" and not c["renormalize"] else M * k * es
        return {"bytes": read + M * k * 8 + M * E * es, "flops": 6 * M * k}
    if c["op"] == "lora":
        K, N, R = c["K"], c["N"], c["R"]
        used = min(c["L"], M)
        return {"bytes": es * (M * K + N * K + used * R * (K + N) + M * N) + 4 * M,
                "flops": 2 * M * (K * N + R * (K + N))}
    H, P = c["H"], M * c["top_k"]
    row, rows = M * H * es, P * H * es
    if c["op"] == "sort":
        tables = 4 * P if c["direction"] == "backward" else 4 * (3 * P + c["E"] + 1)
        return {"bytes": row + rows + tables, "flops": P * H if c["direction"] == "backward" else 0}
    if c["direction"] == "forward":
        return {"bytes": row + rows + 8 * P, "flops": 2 * P * H}
    return {"bytes": row + 2 * rows + 12 * P, "flops": 3 * P * H}


# ------------------------------------------------------------------------- inputs
def _rows(g, n, width, dtype, pad, std=1.0):
    """[n][width] values ~ N(0, std), rows `pad` elements further apart than their width."""
    t = torch.empty(n, width + pad, dtype=dtype, device="cuda")
    t.normal_(0.0, std, generator=g)
    return t[:, :width]


def _routed(c, g):
    """Expert ids of each token's slots: distinct, by Gumbel top-k over even or Zipf(1.2)
    odds; dropped: a share of the pairs is -1, as a capacity limit leaves it."""
    M, E, k = c["M"], c["E"], c["top_k"]
    logp = torch.zeros(E, device="cuda")
    if c["routing"] == "zipf":
        ranks = torch.randperm(E, generator=g, device="cuda") + 1
        logp = -1.2 * torch.log(ranks.float())
    u = torch.rand(M, E, generator=g, device="cuda").clamp_(1e-20, 1.0 - 1e-7)
    ids = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)
    if c["dropped"]:
        ids[torch.rand(M, k, generator=g, device="cuda") < 0.1] = -1
    return ids.contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, dt = c["M"], _DT[c["dtype"]]
    s = {"case": c}
    if c["op"] == "gate":
        E, k = c["E"], c["top_k"]
        logits = torch.randn(M, E, generator=g, device="cuda")
        if c["masked"]:
            logits[torch.rand(M, E, generator=g, device="cuda") < 0.1] = -math.inf
            logits[M // 2] = -math.inf
        s["logits"] = logits.to(dt)
        s["bias"] = None
        if c["scoring"] == "sigmoid":
            s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05
        if c["direction"] == "backward":
            s["dweights"] = torch.randn(M, k, generator=g, device="cuda")
            s["ids"] = _gate_choice(c, s["logits"], s["bias"])[0]
    elif c["op"] == "lora":
        K, N, R, L = c["K"], c["N"], c["R"], c["L"]
        s["x"] = _rows(g, M, K, dt, 0)
        s["w"] = _rows(g, N, K, dt, 0, K ** -0.5)
        s["a"] = _rows(g, L * R, K, dt, 0, K ** -0.5).view(L, R, K)
        s["b"] = _rows(g, L * N, R, dt, 0, R ** -0.5).view(L, N, R)
        s["scales"] = 0.25 + 0.5 * torch.rand(L, generator=g, device="cuda")
        if c["tokens"] == "mixed":  # a request a token; some without an adapter
            ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
            ids[torch.rand(M, generator=g, device="cuda") < 0.1] = -1
        else:  # up to 8 requests of uneven lengths, one after another
            cuts = torch.sort(torch.randint(0, M, (7,), generator=g, device="cuda")).values
            of = torch.randint(-1, L, (8,), generator=g, device="cuda", dtype=torch.int32)
            of[0] = torch.randint(0, L, (1,), generator=g, device="cuda", dtype=torch.int32)[0]
            at = torch.arange(M, device="cuda")
            ids = of[(at[:, None] >= cuts[None]).sum(1)]
        s["ids"] = ids.contiguous()
    else:
        H, k = c["H"], c["top_k"]
        s["ids"] = _routed(c, g)
        if c["op"] == "sort" and c["direction"] == "forward":
            s["x"] = _rows(g, M, H, dt, c["pad"])
        else:
            s["route"] = _route(s["ids"], c["E"])
            s["y"] = _rows(g, M * k, H, dt, c["pad"])
        if c["op"] == "unsort":
            s["weights"] = torch.softmax(torch.randn(M, k, generator=g, device="cuda"), dim=1)
            if c["direction"] == "backward":
                s["dout"] = _rows(g, M, H, dt, c["pad"])
    return s


# -------------------------------------------------------------------- plain forms
def _gate_choice(c, logits, bias):
    """(ids, the chosen experts' choice values): the top_k unmasked experts by choice value,
    ties to the lowest index; empty slots have id -1 and value -inf."""
    M, E = logits.shape
    l = logits.float()
    if c["scoring"] == "softmax":
        choice = l
    else:
        choice = 1.0 / (1.0 + torch.exp(-l)) + bias
    choice = torch.where((l > -math.inf) & (choice > -math.inf), choice, -math.inf)
    G = c["n_group"]
    if G > 1:
        grouped = choice.view(M, G, E // G)
        if c["scoring"] == "softmax":
            score = grouped.amax(-1)
        else:
            score = torch.sort(grouped, dim=-1, descending=True).values[..., :2].sum(-1)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = (best[:, :, None] == torch.arange(G, device=l.device)).any(1)
        choice = torch.where(keep[:, :, None], grouped, -math.inf).view(M, E)
    values, ids = torch.sort(choice, dim=-1, descending=True, stable=True)
    values, ids = values[:, :c["top_k"]], ids[:, :c["top_k"]]
    return torch.where(values > -math.inf, ids, -1).to(torch.int32), values


def _gate_scores(c, logits, ids):
    """The chosen experts' scores and whether each slot holds an expert."""
    l = logits.float()
    there = ids >= 0
    chosen = torch.gather(l, 1, ids.clamp(min=0).long())
    if c["scoring"] == "sigmoid":
        return torch.where(there, 1.0 / (1.0 + torch.exp(-chosen)), 0.0), there
    if c["renormalize"]:
        top = torch.where(there, chosen, -math.inf).amax(1, keepdim=True)
        e = torch.where(there, torch.exp(chosen - top), 0.0)
        return torch.where(there, e / e.sum(1, keepdim=True), 0.0), there
    top = l.amax(1, keepdim=True)
    total = torch.exp(l - top).sum(1, keepdim=True)
    return torch.where(there, torch.exp(chosen - top) / total, 0.0), there


def _gate_plain(s):
    c, logits = s["case"], s["logits"]
    if c["direction"] == "forward":
        ids, _ = _gate_choice(c, logits, s["bias"])
        p, _ = _gate_scores(c, logits, ids)
        if c["scoring"] == "sigmoid" and c["renormalize"]:
            p = p / (p.sum(1, keepdim=True) + 1e-20)
        return {"topk_ids": ids, "topk_weights": p * c["scale"]}
    ids, dw = s["ids"], s["dweights"]
    p, there = _gate_scores(c, logits, ids)
    if c["scoring"] == "softmax":
        # w = scale p: dl = scale p (dw - sum p dw), over the chosen or over all experts
        inner = (p * dw).sum(1, keepdim=True)
        if c["renormalize"]:
            dl = torch.zeros_like(logits, dtype=torch.float32)
        else:
            l = logits.float()
            e = torch.exp(l - l.amax(1, keepdim=True))
            dl = torch.where(there.any(1, keepdim=True),
                             -c["scale"] * inner * e / e.sum(1, keepdim=True), 0.0)
            inner = torch.zeros_like(inner)
        d = c["scale"] * p * (dw - inner)
    else:
        d = c["scale"] * dw
        if c["renormalize"]:
            total = p.sum(1, keepdim=True) + 1e-20
            d = c["scale"] / total * (dw - (p / total * dw).sum(1, keepdim=True))
        d = d * p * (1.0 - p)
        dl = torch.zeros_like(logits, dtype=torch.float32)
    dl = dl.scatter_add(1, ids.clamp(min=0).long(), torch.where(there, d, 0.0))
    return {"dlogits": dl.to(logits.dtype)}


def _route(ids, E):
    """(offsets, sorted_pair, pair_pos) of the pairs in (expert, pair) order."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    at = torch.arange(flat.numel(), device=ids.device)
    pos = torch.empty_like(at)
    pos[order] = at
    return (offsets.to(torch.int32), torch.where(at < offsets[E], order, -1).to(torch.int32),
            torch.where(key < E, pos, -1).to(torch.int32).view(ids.shape))


def _at_pairs(y, pair_pos):
    """[M][k][H] in 32 bits: each pair's row of y, zeros where it has none."""
    rows = y[pair_pos.clamp(min=0).long()].float()
    return torch.where((pair_pos >= 0)[..., None], rows, 0.0)


def _sort_plain(s):
    c = s["case"]
    k = c["top_k"]
    if c["direction"] == "forward":
        offsets, sorted_pair, pair_pos = _route(s["ids"], c["E"])
        rows = s["x"][sorted_pair.clamp(min=0).long() // k]
        xs = torch.where((sorted_pair >= 0)[:, None], rows, 0.0)
        return {"xs": xs, "offsets": offsets, "sorted_pair": sorted_pair, "pair_pos": pair_pos}
    return {"dx": _at_pairs(s["y"], s["route"][2]).sum(1).to(s["y"].dtype)}


def _unsort_plain(s):
    c = s["case"]
    offsets, sorted_pair, pair_pos = s["route"]
    if c["direction"] == "forward":
        out = (s["weights"][..., None] * _at_pairs(s["y"], pair_pos)).sum(1)
        return {"out": out.to(s["y"].dtype)}
    dout = s["dout"].float()
    dw = (_at_pairs(s["y"], pair_pos) * dout[:, None, :]).sum(-1)
    pair = sorted_pair.clamp(min=0).long()
    dy = s["weights"].reshape(-1)[pair][:, None] * dout[pair // c["top_k"]]
    dy = torch.where((sorted_pair >= 0)[:, None], dy, 0.0)
    return {"dy": dy.to(s["y"].dtype), "dweights": dw}


def _lora_plain(s):
    c = s["case"]
    M, N, R, L = c["M"], c["N"], c["R"], c["L"]
    x, ids = s["x"].float(), s["ids"]
    y = x @ s["w"].float().t()
    if M <= L:  # each token's own adapter
        at = ids.clamp(min=0).long()
        t = (s["a"][at].float() @ x[:, :, None])[:, :, 0] * s["scales"][at][:, None]
        delta = (s["b"][at].float() @ t[:, :, None])[:, :, 0]
        y = y + torch.where((ids >= 0)[:, None], delta, 0.0)
    else:  # all adapters, and each token's own kept
        t = (x @ s["a"].float().view(L * R, -1).t()).view(M, L, R) * s["scales"][:, None]
        mine = ids[:, None] == torch.arange(L, device=ids.device)
        t = torch.where(mine[:, :, None], t, 0.0)
        y = y + t.view(M, L * R) @ s["b"].float().transpose(0, 1).reshape(N, L * R).t()
    return {"out": y.to(s["x"].dtype)}


# --------------------------------------------------------------- the library's calls
def _gate_own(s):
    import quantized_moe_grouped_route_gb300 as q
    c = s["case"]
    scoring = q.QMOE_GATE_SIGMOID if c["scoring"] == "sigmoid" else q.QMOE_GATE_SOFTMAX
    if c["direction"] == "forward":
        ids, weights = q.moe_gate(s["logits"], c["top_k"], scoring=scoring, bias=s["bias"],
                                  n_group=c["n_group"], topk_group=c["topk_group"],
                                  renormalize=c["renormalize"], scale=c["scale"])
        return {"topk_ids": ids, "topk_weights": weights}
    return {"dlogits": q.moe_gate_backward(s["dweights"], s["logits"], s["ids"], scoring=scoring,
                                           renormalize=c["renormalize"], scale=c["scale"])}


def _sort_own(s):
    import quantized_moe_grouped_route_gb300 as q
    c = s["case"]
    if c["direction"] == "forward":
        xs, offsets, sorted_pair, pair_pos = q.moe_sort_tokens(s["x"], s["ids"], c["E"])
        return {"xs": xs, "offsets": offsets, "sorted_pair": sorted_pair, "pair_pos": pair_pos}
    return {"dx": q.moe_sort_tokens_backward(s["y"], s["route"][2])}


def _unsort_own(s):
    import quantized_moe_grouped_route_gb300 as q
    offsets, sorted_pair, pair_pos = s["route"]
    if s["case"]["direction"] == "forward":
        return {"out": q.moe_unsort_tokens(s["y"], pair_pos, s["weights"])}
    dy, dw = q.moe_unsort_tokens_backward(s["dout"], s["y"], sorted_pair, pair_pos, s["weights"])
    return {"dy": dy, "dweights": dw}


def _lora_own(s):
    import quantized_moe_grouped_route_gb300 as q
    return {"out": q.qmoe_lora_linear(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scales"])}


_PLAIN = {"gate": _gate_plain, "sort": _sort_plain, "unsort": _unsort_plain, "lora": _lora_plain}
_OWN = {"gate": _gate_own, "sort": _sort_own, "unsort": _unsort_own, "lora": _lora_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The floating outputs from the operators' definitions in 64 bits, expert by expert,
    slot by slot and adapter by adapter."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "gate":
        return _exact_gate(c, s)
    if c["op"] == "lora":
        x = s["x"].double()
        y = x @ s["w"].double().t()
        for a in range(c["L"]):
            rows = (s["ids"] == a).nonzero()[:, 0]
            if rows.numel():
                t = x[rows] @ s["a"][a].double().t()
                y[rows] += s["scales"][a].double() * (t @ s["b"][a].double().t())
        return {"out": y}
    ids, k = s["ids"], c["top_k"]
    flat = ids.reshape(-1)
    pairs = torch.cat([(flat == e).nonzero()[:, 0] for e in range(c["E"])])  # in sorted order
    n = pairs.numel()
    if c["op"] == "sort" and c["direction"] == "forward":
        xs = torch.zeros(flat.numel(), c["H"], dtype=torch.float64, device="cuda")
        xs[:n] = s["x"].double()[pairs // k]
        return {"xs": xs, "offsets": None, "sorted_pair": None, "pair_pos": None}
    where = torch.full_like(flat, -1, dtype=torch.int64)
    where[pairs] = torch.arange(n, device="cuda")
    where = where.view(-1, k)
    if c["op"] == "unsort" and c["direction"] == "backward":
        dout, w = s["dout"].double(), s["weights"].double().reshape(-1)
        dy = torch.zeros(flat.numel(), c["H"], dtype=torch.float64, device="cuda")
        dy[:n] = w[pairs][:, None] * dout[pairs // k]
        dw = torch.zeros(where.shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            m = (where[:, j] >= 0).nonzero()[:, 0]
            dw[m, j] = (dout[m] * s["y"][where[m, j]].double()).sum(1)
        return {"dy": dy, "dweights": dw}
    out = torch.zeros(c["M"], c["H"], dtype=torch.float64, device="cuda")
    for j in range(k):
        m = (where[:, j] >= 0).nonzero()[:, 0]
        row = s["y"][where[m, j]].double()
        out[m] += row if c["op"] == "sort" else s["weights"][m, j].double()[:, None] * row
    return {"dx": out} if c["op"] == "sort" else {"out": out}


def _exact_gate(c, s):
    l = s["logits"].double()
    # which experts: the definition's choice values are in 32 bits, so they are taken as such
    ids = s["ids"] if c["direction"] == "backward" else _gate_choice(c, s["logits"], s["bias"])[0]
    hot = torch.zeros(c["M"], c["E"], dtype=torch.bool, device="cuda")
    m, j = (ids >= 0).nonzero(as_tuple=True)
    hot[m, ids[m, j].long()] = True
    hot = hot & ~torch.isinf(l)
    l = l.clone().requires_grad_(True)
    if c["scoring"] == "sigmoid":
        p = torch.sigmoid(l)
        if c["renormalize"]:
            p = p / ((p * hot).sum(1, keepdim=True) + 1e-20)
    else:
        seen = hot if c["renormalize"] else l.detach() > -math.inf
        e = torch.where(seen, l, -1e9)
        p = torch.softmax(e, 1)
    w = torch.where(hot, p * c["scale"], 0.0)
    w = torch.where(ids >= 0, torch.gather(w, 1, ids.clamp(min=0).long()), 0.0)
    if c["direction"] == "forward":
        return {"topk_ids": None, "topk_weights": w.detach()}
    (w * s["dweights"].double()).sum().backward()
    return {"dlogits": torch.nan_to_num(l.grad)}
