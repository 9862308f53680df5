"""Routing, rows and products of a routed layer of any number of tokens, in their plain form and as the library's calls.

Three operators, with their gradients:

``topk``     the k experts of each token and their gating weights from the router's logits: with S the k largest
             logits (ties to the lower index), w_e = g_e / sum_S g, g = exp(l) or sigma(l); not renormalised, softmax
             divides by the sum over all experts and sigmoid by nothing.  Back: the weights' gradient to the logits
``rows``     token rows to their places in the order by expert and back: xs[pos[t, s]] = x[t];
             y[t] = addend[t] + sum_s w[t, s] o[pos[t, s]].  Back: do[pos[t, s]] = w[t, s] dy[t],
             dw[t, s] = <o[pos[t, s]], dy[t]>
``product``  v_i = x[row_i] w_g^T + bias_g for the places i of each group g (an expert; one group is a plain product),
             y = act(v) + residual.  swiglu: v has 2 N columns, gate then up, act(v) = silu(gate) up.  Back:
             (dy w_g) act'(z), the matrices taken as [K, N]

``run`` is one pass through an operator.  Where ``own`` is false it is written in elementary torch operations in
32 bits; where it is true it makes the library's calls.  ``exact`` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode batch over 128 experts: latency
        {"name": "topk_decode", "op": "topk", "back": False, "T": 16, "E": 128, "k": 8, "gating": "softmax",
         "renormalize": True, "type": "fp32", "padded": 2},
        # a training batch of a sigmoid router over 256 experts, with a ragged end
        {"name": "topk_batch", "op": "topk", "back": False, "T": 65536, "E": 256, "k": 8, "gating": "sigmoid",
         "renormalize": True, "type": "fp32", "padded": 777},
        # its way back for a softmax router whose weights keep the sum over all experts: the whole row has a gradient,
        # which is added to that of the balance loss
        {"name": "topk_back", "op": "topk", "back": True, "T": 65536, "E": 128, "k": 8, "gating": "softmax",
         "renormalize": False, "type": "bf16", "padded": 777},
        # a decode batch's expert outputs onto the residual stream: latency
        {"name": "combine_decode", "op": "rows", "way": "combine", "T": 16, "k": 8, "E": 128, "n": 4096,
         "type": "bf16", "out": "fp32", "weights": True, "addend": True, "padded": 2},
        # a prefill chunk's expert outputs
        {"name": "combine_prefill", "op": "rows", "way": "combine", "T": 8192, "k": 8, "E": 128, "n": 4096,
         "type": "bf16", "out": "bf16", "weights": True, "addend": False, "padded": 0},
        # the way back of a training batch, odd in its tokens
        {"name": "combine_back", "op": "rows", "way": "combine_grad", "T": 8191, "k": 4, "E": 32, "n": 2880,
         "type": "bf16", "out": "bf16", "weights": True, "addend": False, "padded": 7},
        # a prefill chunk's rows to their places, the widest layer
        {"name": "dispatch_prefill", "op": "rows", "way": "dispatch", "T": 4096, "k": 8, "E": 256, "n": 7168,
         "type": "bf16", "out": "bf16", "weights": False, "addend": False, "padded": 100},
        # one token through the gate and up matrices of its 8 of 256 experts: weight bandwidth, latency
        {"name": "product_token", "op": "product", "T": 1, "k": 8, "E": 256, "N": 512, "K": 2048, "act": "swiglu",
         "bias": False, "residual": False, "keep": False, "gather": True, "out": "bf16"},
        # a decode batch through the down matrices of 32 experts with biases: nearly all are read for two rows
        {"name": "product_decode", "op": "product", "T": 16, "k": 4, "E": 32, "N": 2880, "K": 2880, "act": "none",
         "bias": True, "residual": False, "keep": False, "gather": False, "out": "bf16"},
        # the way back of a short training step through the down matrices and the gated activation, ragged
        {"name": "product_back", "op": "product", "T": 777, "k": 4, "E": 32, "N": 2880, "K": 2880,
         "act": "swiglu_grad", "bias": False, "residual": False, "keep": False, "gather": False, "out": "bf16"},
        # a prefill chunk through a shared expert's down matrix, added to the residual stream
        {"name": "product_dense", "op": "product", "T": 8192, "k": 1, "E": 1, "N": 7168, "K": 2048, "act": "none",
         "bias": False, "residual": True, "keep": False, "gather": False, "out": "fp32"},
        # a training batch through the gate and up matrices of 32 experts with biases, gathered, what the activation
        # takes kept for the way back; odd in its tokens
        {"name": "product_prefill", "op": "product", "T": 8191, "k": 4, "E": 32, "N": 2880, "K": 2880,
         "act": "swiglu", "bias": True, "residual": False, "keep": True, "gather": True, "out": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "rows", "product", "product"])
    if op == "topk":
        E = _spread(rng, 8, 512)
        k = rng.randint(1, 8)
        T = _spread(rng, 1, min(65536, 65536 * 256 // E))
        return {"op": op, "back": rng.random() < 0.5, "T": T, "E": E, "k": k,
                "gating": rng.choice(["softmax", "sigmoid"]), "renormalize": rng.random() < 0.6,
                "type": rng.choice(["fp32", "bf16"]), "padded": rng.randint(0, T // 8)}
    if op == "rows":
        n = _spread(rng, 64, 7168)
        if rng.random() < 0.7:
            n = max(8, n // 8 * 8)
        E = _spread(rng, 8, 256)
        k = rng.randint(1, 8)
        T = _spread(rng, 1, max(1, min(16384, 8192 * 4096 * 4 // (n * k))))
        return {"op": op, "way": rng.choice(["dispatch", "combine", "combine_grad"]), "T": T, "k": k, "E": E, "n": n,
                "type": rng.choice(["fp32", "bf16"]), "out": rng.choice(["fp32", "bf16"]),
                "weights": rng.random() < 0.7, "addend": rng.random() < 0.5, "padded": rng.randint(0, T // 8)}
    act = rng.choice(["none", "none", "silu", "gelu", "swiglu", "swiglu", "silu_grad", "gelu_grad", "swiglu_grad"])
    back = act.endswith("_grad")
    K = 8 * _spread(rng, 8, 896)
    N = _spread(rng, 64, 4096)
    if back:
        N = max(8, N // 8 * 8)
    if act == "swiglu":
        N = max(16, N // 16 * 16)
    wide = 2 if act == "swiglu" else 1
    if rng.random() < 0.4:
        E, k = 1, 1
        T = _spread(rng, 1, max(1, min(8192, 2 ** 38 // (N * wide * K))))
    else:
        E = _spread(rng, 2, max(2, min(128, 2 ** 30 // (N * wide * K))))
        k = rng.randint(1, min(8, E))
        T = _spread(rng, 1, max(1, min(8192, 2 ** 38 // (N * wide * K * k))))
    return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "act": act, "bias": not back and rng.random() < 0.5,
            "residual": not back and rng.random() < 0.4, "keep": not back and act != "none" and rng.random() < 0.4,
            "gather": not back and E > 1 and rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "fp32"])}


# ----------------------------------------------------------------- inputs

def _hidden(T, n, gen, scale=1.0):
    """Hidden states: normal values with a few large channels, as residual streams have them."""
    gain = torch.ones(n, device="cuda")
    gain[torch.randint(0, n, (max(1, n // 200),), device="cuda", generator=gen)] = 12.0
    return torch.randn(T, n, device="cuda", generator=gen) * gain * scale


def _logits(T, E, gen):
    """Router logits: some experts are liked better than others."""
    return torch.randn(T, E, device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)


def _largest(logits, k):
    """Ids of the k largest of each row, ties to the lower index."""
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]


def _ids(T, k, E, padded, gen):
    ids = _largest(_logits(T, E, gen), k).to(torch.int32)
    if padded:
        ids[T - padded:] = -1
    return ids.contiguous()


def _sorted(ids, E):
    """counts [E], offsets [E + 1], rows [T k] and pos [T, k] of a routing, and how many pairs take part."""
    T, k = ids.shape
    key = ids.reshape(-1).long()
    key = torch.where(key < 0, torch.full_like(key, E), key)
    by = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=key.device).index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    place = torch.arange(T * k, device=key.device)
    live = place < offsets[E]
    pos = torch.empty_like(by)
    pos[by] = torch.where(live, place, torch.full_like(place, -1))
    rows = torch.where(live, by // k, torch.full_like(by, -1))
    return counts, offsets.to(torch.int32), rows.to(torch.int32), pos.reshape(T, k).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 29)
    s = {"case": dict(case)}
    op, T = case["op"], case["T"]
    new = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    if op == "topk":
        E, dt = case["E"], TYPES[case["type"]]
        k = min(case["k"], E)
        s["logits"] = _logits(T, E, gen).to(dt)
        s["valid"] = new(T, dtype=torch.uint8)
        s["valid"][:T - case["padded"]] = 1
        if case["back"]:
            s["ids"] = _largest(s["logits"], k).to(torch.int32).contiguous()
            s["ids"][T - case["padded"]:] = -1
            s["dweights"] = rand(T, k)
            s["addend"] = (0.05 * rand(T, E)).to(dt)      # the balance loss's
            s["dlogits"] = new(T, E, dtype=dt)
        else:
            s["ids"], s["weights"] = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
    elif op == "rows":
        k, E, n, dt, out = min(case["k"], case["E"]), case["E"], case["n"], TYPES[case["type"]], TYPES[case["out"]]
        s["pos"] = _sorted(_ids(T, k, E, case["padded"], gen), E)[3]
        if case["way"] == "dispatch":
            s["x"], s["xs"] = _hidden(T, n, gen).to(dt), new(T * k, n, dtype=dt)
        else:
            s["weights"] = torch.softmax(rand(T, k), 1) if case["weights"] else None
            s["o"] = _hidden(T * k, n, gen, 0.3).to(dt)
            if case["way"] == "combine":
                s["addend"] = _hidden(T, n, gen).to(out) if case["addend"] else None
                s["y"] = new(T, n, dtype=out)
            else:
                s["dy"] = rand(T, n).to(out)
                s["do"], s["dweights"] = new(T * k, n, dtype=dt), new(T, k, dtype=torch.float32)
    else:
        k, E, N, K, act, out = case["k"], case["E"], case["N"], case["K"], case["act"], TYPES[case["out"]]
        back = act.endswith("_grad")
        wide = 2 * N if act == "swiglu" else N
        M = T * k
        s["w"] = torch.empty((E, K, N) if back else (E, wide, K), dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            s["w"][e] = rand(*s["w"].shape[1:]) * K ** -0.5
        s["rows"] = s["offsets"] = s["group"] = None
        if E > 1:
            counts, s["offsets"], rows, _ = _sorted(_ids(T, k, E, 0, gen), E)
            s["cap"] = int(counts.max())
            s["group"] = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
            s["at"] = torch.arange(M, device="cuda") - s["offsets"].long()[s["group"]]
            if case["gather"]:
                s["rows"] = rows
        else:
            s["w"] = s["w"][0]
        x = rand(M, K) if back else _hidden(T if s["rows"] is not None else M, K, gen)
        s["x"] = x.to(torch.bfloat16)
        s["bias"] = 0.3 * rand(*((E,) if E > 1 else ()), wide) if case["bias"] else None
        s["residual"] = _hidden(M, N, gen).to(out) if case["residual"] else None
        s["y"] = new(M, 2 * N if act == "swiglu_grad" else N, dtype=out)
        s["z"] = new(M, wide, dtype=out) if case["keep"] else None
        if back:
            s["z"] = (1.5 * rand(M, 2 * N if act == "swiglu_grad" else N)).to(out)
        if own:
            import quantized_routed_expert_router_gb300 as moe
            s["ws"] = new(moe.moe_matmul_workspace_bytes(), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    if own:
        return _own(s)
    return {"topk": _topk, "rows": _rows, "product": _product}[s["case"]["op"]](s)


def _own(s):
    import quantized_routed_expert_router_gb300 as moe
    case = s["case"]
    if case["op"] == "topk":
        gating = moe.SOFTMAX if case["gating"] == "softmax" else moe.SIGMOID
        if case["back"]:
            moe.moe_topk_grad(s["logits"], s["ids"], s["dweights"], gating, case["renormalize"], s["dlogits"],
                              addend=s["addend"])
            return {"dlogits": s["dlogits"]}
        moe.moe_topk(s["logits"], gating, case["renormalize"], s["ids"], s["weights"], valid=s["valid"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if case["op"] == "rows":
        if case["way"] == "dispatch":
            moe.moe_dispatch_rows(s["x"], s["pos"], s["xs"])
            return {"xs": s["xs"]}
        if case["way"] == "combine":
            moe.moe_combine_rows(s["o"], s["pos"], s["y"], weights=s["weights"], addend=s["addend"])
            return {"y": s["y"]}
        moe.moe_combine_grad(s["dy"], s["pos"], weights=s["weights"], o=s["o"], do=s["do"], dweights=s["dweights"])
        return {"do": s["do"], "dweights": s["dweights"]}
    act = {"none": moe.ACT_NONE, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "swiglu": moe.ACT_SWIGLU,
           "silu_grad": moe.ACT_SILU_GRAD, "gelu_grad": moe.ACT_GELU_GRAD,
           "swiglu_grad": moe.ACT_SWIGLU_GRAD}[case["act"]]
    back = case["act"].endswith("_grad")
    moe.moe_matmul(s["x"], s["w"], s["y"], s["ws"], act=act, bias=s["bias"], residual=s["residual"], z=s["z"],
                   offsets=s["offsets"], rows=s["rows"], transposed=back)
    return {"y": s["y"], "z": s["z"]} if case["keep"] else {"y": s["y"]}


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _topk(s):
    case, l = s["case"], s["logits"].float()
    soft, renorm = case["gating"] == "softmax", case["renormalize"]
    if soft:
        e = torch.exp(l - l.amax(1, keepdim=True))
        g = e if renorm else e / e.sum(1, keepdim=True)
    else:
        g = _sigmoid(l)
    if not case["back"]:
        ids = _largest(l, s["ids"].shape[1])
        w = torch.gather(g, 1, ids)
        if renorm:
            w = w / w.sum(1, keepdim=True)
        live = s["valid"].bool()[:, None]
        ids = torch.where(live, ids, torch.full_like(ids, -1)).to(torch.int32)
        return {"ids": ids, "weights": torch.where(live, w, torch.zeros_like(w))}
    live = (s["ids"] >= 0).float()
    ids = s["ids"].long().clamp(min=0)
    dw = s["dweights"] * live
    w = torch.gather(g, 1, ids)
    slope = 1.0 if soft else 1.0 - w
    if renorm:
        w = w / w.sum(1, keepdim=True)
    if renorm or soft:
        dot = (w * dw).sum(1, keepdim=True)
    if soft and not renorm:
        grad = -g * dot
        grad.scatter_add_(1, ids, w * dw)
    else:
        d = slope * w * ((dw - dot) * live if renorm else dw)
        grad = torch.zeros_like(l).scatter_add_(1, ids, d)
    return {"dlogits": (s["addend"].float() + grad).to(s["logits"].dtype)}


def _rows(s):
    case, pos = s["case"], s["pos"].long()
    T, k = pos.shape
    live = pos >= 0
    if case["way"] == "dispatch":
        xs = torch.zeros_like(s["xs"])
        xs[pos[live]] = s["x"][:, None, :].expand(T, k, -1)[live]
        return {"xs": xs}
    w = s["weights"] if s["weights"] is not None else torch.ones(T, k, device=pos.device)
    w = w * live
    if case["way"] == "combine":
        y = s["addend"].float() if s["addend"] is not None else torch.zeros(T, case["n"], device=pos.device)
        for i in range(k):
            y = y + w[:, i:i + 1] * s["o"][pos[:, i].clamp(min=0)].float()
        return {"y": y.to(s["y"].dtype)}
    dy = s["dy"].float()
    do, dw = torch.zeros_like(s["do"]), torch.zeros_like(s["dweights"])
    for i in range(k):
        at = pos[:, i][live[:, i]]
        do[at] = (w[:, i:i + 1] * dy)[live[:, i]].to(do.dtype)
        dw[:, i] = (s["o"][pos[:, i].clamp(min=0)].float() * dy).sum(1) * live[:, i]
    return {"do": do, "dweights": dw}


def _slope(act, z):
    """act'(z)"""
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    g = _sigmoid(z)
    return g * (1.0 + z * (1.0 - g))


def _product(s):
    case, act, N, out = s["case"], s["case"]["act"], s["case"]["N"], s["y"].dtype
    x, w = s["x"].float(), s["w"].float()
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    if not act.endswith("_grad"):
        w = w.transpose(-1, -2)
    if s["group"] is None:
        v = x @ w
    else:
        xs = torch.zeros(w.shape[0], s["cap"], x.shape[1], device=x.device)
        xs[s["group"], s["at"]] = x
        v = torch.bmm(xs, w)[s["group"], s["at"]]
    if s["bias"] is not None:
        v = v + (s["bias"] if s["group"] is None else s["bias"][s["group"]])
    if act == "none":
        y = v
    elif act == "silu":
        y = v * _sigmoid(v)
    elif act == "gelu":
        y = v * 0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5))
    elif act == "swiglu":
        y = v[:, :N] * _sigmoid(v[:, :N]) * v[:, N:]
    elif act == "swiglu_grad":
        z = s["z"].float()
        y = torch.cat([v * z[:, N:] * _slope("silu", z[:, :N]), v * z[:, :N] * _sigmoid(z[:, :N])], 1)
    else:
        y = v * _slope(act[:-5], s["z"].float())
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(out), "z": v.to(out)} if case["keep"] else {"y": y.to(out)}


# ------------------------------------------------------------------- work

def work(case):
    op, T = case["op"], case["T"]
    if op == "topk":
        E, k, b = case["E"], min(case["k"], case["E"]), BYTES[case["type"]]
        if not case["back"]:
            return {"bytes": T * (E * b + 8 * k + 1), "flops": 4 * T * E}
        seen = E if case["gating"] == "softmax" and not case["renormalize"] else k     # logits that are looked at
        return {"bytes": T * (seen * b + 2 * E * b + 8 * k), "flops": 6 * T * seen}
    if op == "rows":
        k, n, b, o = min(case["k"], case["E"]), case["n"], BYTES[case["type"]], BYTES[case["out"]]
        pairs = (T - case["padded"]) * k
        idx = 4 * T * k
        if case["way"] == "dispatch":
            return {"bytes": (T - case["padded"]) * n * b + pairs * n * b + idx, "flops": 0}
        idx += 4 * T * k if case["weights"] else 0
        if case["way"] == "combine":
            return {"bytes": pairs * n * b + T * n * o * (2 if case["addend"] else 1) + idx, "flops": 2 * pairs * n}
        return {"bytes": (T - case["padded"]) * n * o + 2 * pairs * n * b + idx + 4 * T * k, "flops": 3 * pairs * n}
    k, E, N, K, o = case["k"], case["E"], case["N"], case["K"], BYTES[case["out"]]
    M, act = T * k, case["act"]
    wide = 2 * N if act == "swiglu" else N
    hit = 1 if E == 1 else E * (1 - (1 - k / E) ** T)     # experts that some token chose
    outs = M * (2 * N if act == "swiglu_grad" else N) * o
    ins = M * N * o if case["residual"] else 0
    if act.endswith("_grad"):
        ins += outs
    if case["keep"]:
        outs += M * wide * o
    if case["bias"]:
        ins += hit * wide * 4
    return {"bytes": (T if case["gather"] else M) * K * 2 + hit * wide * K * 2 + ins + outs,
            "flops": 2 * M * wide * K}


# ------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"topk": _exact_topk, "rows": _exact_rows, "product": _exact_product}[case["op"]](case, s)


def _gating(l, chosen, case):
    """Gating weights of the chosen experts, a function of the logits that autograd can follow."""
    log = torch.log_softmax(l, 1) if case["gating"] == "softmax" else torch.nn.functional.logsigmoid(l)
    log = torch.gather(log, 1, chosen)
    return torch.exp(log - torch.logsumexp(log, 1, keepdim=True) if case["renormalize"] else log)


def _exact_topk(case, s):
    l = s["logits"].double()
    if not case["back"]:
        weights = _gating(l, _largest(l, s["ids"].shape[1]), case)
        weights[~s["valid"].bool()] = 0
        return {"ids": None, "weights": weights}      # whole numbers: nothing is rounded
    l.requires_grad_(True)
    live = s["valid"].double()[:, None]
    value = (_gating(l, s["ids"].long().clamp(min=0), case) * s["dweights"].double() * live).sum()
    return {"dlogits": torch.autograd.grad(value, l)[0] + s["addend"].double()}


def _exact_rows(case, s):
    pos = s["pos"].long()
    T, k = pos.shape
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[pos >= 0]
    place = pos[pos >= 0]
    if case["way"] == "dispatch":
        out = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda")
        return {"xs": out.index_copy_(0, place, s["x"].double()[token])}
    n = case["n"]
    w = s["weights"].double()[pos >= 0] if s["weights"] is not None else torch.ones(len(place), device="cuda").double()
    if case["way"] == "combine":
        y = torch.zeros(T, n, dtype=torch.float64, device="cuda") if s["addend"] is None else s["addend"].double()
        return {"y": y.index_add_(0, token, w[:, None] * s["o"].double()[place])}
    do = torch.zeros(s["do"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dy = s["dy"].double()
    do.index_copy_(0, place, w[:, None] * dy[token])
    dw[pos >= 0] = torch.linalg.vecdot(s["o"].double()[place], dy[token])
    return {"do": do, "dweights": dw}


def _exact_product(case, s):
    act, N, E = case["act"], case["N"], case["E"]
    M, K = case["T"] * case["k"], case["K"]
    wide = 2 * N if act == "swiglu" else N
    if 2 * M * wide * K > 4e12:
        return {"y": None, "z": None} if case["keep"] else {"y": None}
    w = s["w"] if E > 1 else s["w"][None]
    v = torch.zeros(M, wide, dtype=torch.float64, device="cuda")
    ends = [0, M] if E == 1 else s["offsets"].tolist()
    for g in range(E):
        a, b = ends[g], ends[g + 1]
        if a == b:
            continue
        x = s["x"][a:b] if s["rows"] is None else s["x"][s["rows"][a:b].long()]
        v[a:b] = torch.einsum("ik,kn->in" if act.endswith("_grad") else "ik,nk->in", x.double(), w[g].double())
        if s["bias"] is not None:
            v[a:b] += (s["bias"] if E == 1 else s["bias"][g]).double()
    f = torch.nn.functional
    if act.endswith("_grad"):
        z = s["z"].double().requires_grad_(True)
        if act == "swiglu_grad":
            h = f.silu(z[:, :N]) * z[:, N:]
        else:
            h = f.silu(z) if act == "silu_grad" else f.gelu(z)
        y = torch.autograd.grad(h, z, v)[0]
    elif act == "swiglu":
        y = f.silu(v[:, :N]) * v[:, N:]
    else:
        y = {"none": lambda t: t.clone(), "silu": f.silu, "gelu": f.gelu}[act](v)
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y, "z": v} if case["keep"] else {"y": y}
