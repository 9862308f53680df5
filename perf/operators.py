"""The operators around the routed experts, in their plain form and as the library's calls.

Four operators:

``norm``     residual addition, root-mean-square norm and 8-bit rows with a scale for each 128 values:
             s = x + residual, v = s / sqrt(mean(s^2) + eps) * weight, scale = max|v| / 448 over a group,
             x8 = e4m3(v / scale)
``order``    the (token, slot) pairs of a routing sorted by expert, tokens in order within an expert: counts,
             offsets, the token of each sorted place and the sorted place of each pair
``balance``  the router's balance loss and its gradient: with p the gate probabilities of a token, c the
             experts' counts and N = sum(c):  loss = alpha E k / N^2 sum_t sum_e c_e p_te
``matmul``   y_i = sum_b x_scale[row_i, b] w_scale[g, n/128, b] sum_(k in block b) x8[row_i, k] w[g, n, k]
             for the rows i of each group g (a group is an expert; one group is a plain dense product)

``run`` is one pass through an operator.  Where ``own`` is false it is written in elementary torch operations in
32 bits; where it is true it makes the library's calls.  ``exact`` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

FP8_MAX = 448.0
GROUP = 128
EPS = 1e-6
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token of the widest layer: latency
        {"name": "norm_token", "op": "norm", "T": 1, "n": 7168, "type": "fp32"},
        # a prefill chunk of that layer: bandwidth
        {"name": "norm_prefill", "op": "norm", "T": 8192, "n": 7168, "type": "bf16"},
        # a decode batch over 128 experts, two of its tokens padding
        {"name": "order_decode", "op": "order", "T": 16, "k": 8, "E": 128, "padded": 2},
        # a training batch over 256 experts, with a ragged end
        {"name": "order_batch", "op": "order", "T": 65536, "k": 8, "E": 256, "padded": 777},
        # a small softmax router step with an odd token count
        {"name": "balance_small", "op": "balance", "T": 509, "k": 4, "E": 32, "gating": "softmax", "type": "fp32",
         "padded": 9},
        # a training batch of a sigmoid router over 256 experts
        {"name": "balance_batch", "op": "balance", "T": 65536, "k": 8, "E": 256, "gating": "sigmoid", "type": "fp32",
         "padded": 777},
        # one token through a shared expert's gate matrix: weight bandwidth, latency
        {"name": "matmul_token", "op": "matmul", "T": 1, "k": 1, "E": 1, "N": 2048, "K": 7168, "type": "bf16"},
        # a decode batch through a shared expert's down matrix, fp32 result as the residual stream takes it
        {"name": "matmul_batch", "op": "matmul", "T": 16, "k": 1, "E": 1, "N": 7168, "K": 2048, "type": "fp32"},
        # a decode batch over 128 experts: nearly every expert is read for one row or two
        {"name": "matmul_experts_decode", "op": "matmul", "T": 16, "k": 8, "E": 128, "N": 1536, "K": 4096,
         "type": "bf16"},
        # a short prefill over 32 experts, width and depth no multiple of 128
        {"name": "matmul_experts_ragged", "op": "matmul", "T": 777, "k": 4, "E": 32, "N": 2880, "K": 2880,
         "type": "bf16"},
        # a prefill chunk over 128 experts
        {"name": "matmul_experts_prefill", "op": "matmul", "T": 8192, "k": 8, "E": 128, "N": 1536, "K": 4096,
         "type": "bf16"},
        # a prefill chunk through a shared expert's gate matrix
        {"name": "matmul_prefill", "op": "matmul", "T": 8192, "k": 1, "E": 1, "N": 2048, "K": 7168, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "order", "balance", "matmul", "matmul"])
    if op == "norm":
        n = 16 * _spread(rng, 16, 512)
        T = _spread(rng, 1, max(1, min(16384, 8192 * 7168 // n)))
        return {"op": op, "T": T, "n": n, "type": rng.choice(["fp32", "bf16"]) if T * n < 8192 * 3584 else "bf16"}
    if op in ("order", "balance"):
        E = _spread(rng, 8, 256)
        k = rng.randint(1, 8)
        T = _spread(rng, 1, 65536)
        case = {"op": op, "T": T, "k": k, "E": E, "padded": rng.randint(0, T // 8)}
        if op == "balance":
            case.update(gating=rng.choice(["softmax", "sigmoid"]), type=rng.choice(["fp32", "bf16"]))
        return case
    K = 16 * _spread(rng, 16, 448)
    N = _spread(rng, 256, 7168)
    if rng.random() < 0.7:
        N = max(8, N // 8 * 8)
    if rng.random() < 0.4:
        E, k = 1, 1
        T = _spread(rng, 1, max(1, min(8192, 8192 * 7168 * 2048 // (N * K))))
    else:
        E = _spread(rng, 2, max(2, min(128, 128 * 1536 * 4096 // (N * K))))
        k = rng.randint(1, min(8, E))
        T = _spread(rng, 1, max(1, min(8192, 32768 * 1536 * 4096 // (N * K * k))))
    return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "type": rng.choice(["bf16", "bf16", "fp32"])}


# ----------------------------------------------------------------- inputs

def _hidden(T, n, gen, scale=1.0):
    """Hidden states: normal values with a few large channels, as residual streams have them."""
    gain = torch.ones(n, device="cuda")
    gain[torch.randint(0, n, (max(1, n // 200),), device="cuda", generator=gen)] = 12.0
    return torch.randn(T, n, device="cuda", generator=gen) * gain * scale


def _routing(T, k, E, padded, gen, logits=None):
    """Expert ids of T tokens; some experts are liked better than others, the padded tokens at the end have -1."""
    if logits is None:
        logits = torch.randn(T, E, device="cuda", generator=gen)
        logits += 0.3 * torch.randn(E, device="cuda", generator=gen)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    if padded:
        ids[T - padded:] = -1
    return ids.contiguous()


def _sorted(ids, E):
    """counts [E], offsets [E + 1], rows [T k], pos [T, k] of a routing."""
    T, k = ids.shape
    key = ids.reshape(-1).long()
    key = torch.where((key < 0) | (key >= E), torch.full_like(key, E), key)
    by = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0) if key.numel() * E < 1 << 24 else \
        torch.zeros(E + 1, dtype=torch.int64, device=key.device).index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    place = torch.arange(T * k, device=key.device)
    live = place < offsets[E]
    rows = torch.where(live, by // k, torch.full_like(by, -1))
    pos = torch.empty_like(by)
    pos[by] = torch.where(live, place, torch.full_like(place, -1))
    i32 = torch.int32
    return counts.to(i32), offsets.to(i32), rows.to(i32), pos.reshape(T, k).to(i32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 17)
    s = {"case": dict(case)}
    op, T = case["op"], case["T"]
    new = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "norm":
        n, dt = case["n"], TYPES[case["type"]]
        s["x"] = _hidden(T, n, gen, 0.5).to(dt)
        s["residual"] = _hidden(T, n, gen).to(dt)
        s["weight"] = 1.0 + 0.2 * torch.randn(n, device="cuda", generator=gen)
        s["residual_out"] = new(T, n, dtype=dt)
        s["y"] = new(T, n, dtype=dt)
        s["x8"] = new(T, n, dtype=torch.float8_e4m3fn)
        s["x8_scale"] = new(T, -(-n // GROUP), dtype=torch.float32)
    elif op == "order":
        k, E = case["k"], case["E"]
        s["ids"] = _routing(T, min(k, E), E, case["padded"], gen)
        k = s["ids"].shape[1]
        s["counts"], s["offsets"] = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32)
        s["rows"], s["pos"] = new(T * k, dtype=torch.int32), new(T, k, dtype=torch.int32)
        if own:
            import quantized_routed_expert_router_gb300 as moe
            s["ws"] = new(max(16, moe.moe_expert_order_workspace_bytes(T, k, E)), dtype=torch.uint8)
    elif op == "balance":
        k, E, dt = min(case["k"], case["E"]), case["E"], TYPES[case["type"]]
        logits = torch.randn(T, E, device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)
        s["logits"] = logits.to(dt)
        ids = _routing(T, k, E, case["padded"], gen, logits)
        s["counts"] = _sorted(ids, E)[0]
        s["valid"] = (ids[:, 0] >= 0).to(torch.uint8)
        s["k"], s["alpha"] = k, 0.01
        s["grad_loss"] = torch.rand(1, device="cuda", generator=gen) + 0.5
        s["loss"], s["dlogits"] = new(1, dtype=torch.float32), new(T, E, dtype=dt)
        if own:
            import quantized_routed_expert_router_gb300 as moe
            s["ws"] = new(moe.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8)
    else:
        k, E, N, K = case["k"], case["E"], case["N"], case["K"]
        kb, nb = -(-K // GROUP), -(-N // GROUP)
        x = _hidden(T, K, gen)
        pad = torch.nn.functional.pad(x, (0, kb * GROUP - K)).reshape(T, kb, GROUP)
        s["x_scale"] = (pad.abs().amax(2) / FP8_MAX).contiguous()
        s["x8"] = (pad / s["x_scale"][:, :, None]).reshape(T, kb * GROUP)[:, :K].contiguous().to(torch.float8_e4m3fn)
        s["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            w = torch.randn(N, K, device="cuda", generator=gen) * 110.0
            s["w"][e] = w.clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s["w_scale"] = (0.5 + torch.rand(E, nb, kb, device="cuda", generator=gen)) * (0.02 / 110.0)
        if E == 1:
            s["w"], s["w_scale"] = s["w"][0], s["w_scale"][0]
            s["rows"] = s["offsets"] = None
        else:
            ids = _routing(T, k, E, 0, gen)
            counts, s["offsets"], s["rows"], _ = _sorted(ids, E)
            s["cap"] = int(counts.max())
            group = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
            s["group"], s["at"] = group, torch.arange(T * k, device="cuda") - s["offsets"].long()[group]
        s["y"] = new(T * k, N, dtype=TYPES[case["type"]])
        if own:
            import quantized_routed_expert_router_gb300 as moe
            s["ws"] = new(moe.moe_fp8_matmul_workspace_bytes(), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return {"norm": _norm, "order": _order, "balance": _balance, "matmul": _matmul}[op](s)


def _own(s):
    import quantized_routed_expert_router_gb300 as moe
    op = s["case"]["op"]
    if op == "norm":
        moe.moe_add_rmsnorm(s["x"], s["residual"], s["weight"], EPS, residual_out=s["residual_out"], y=s["y"],
                            x8=s["x8"], x8_scale=s["x8_scale"])
        return {"residual": s["residual_out"], "y": s["y"], "x8": s["x8"], "scale": s["x8_scale"]}
    if op == "order":
        moe.moe_expert_order(s["ids"], s["case"]["E"], s["ws"], counts=s["counts"], offsets=s["offsets"],
                             rows=s["rows"], pos=s["pos"])
        return {"counts": s["counts"], "offsets": s["offsets"], "rows": s["rows"], "pos": s["pos"]}
    if op == "balance":
        gating = moe.SOFTMAX if s["case"]["gating"] == "softmax" else moe.SIGMOID
        moe.moe_balance_loss(s["logits"], s["counts"], s["k"], gating, s["alpha"], s["ws"], valid=s["valid"],
                             grad_loss=s["grad_loss"], loss=s["loss"], dlogits=s["dlogits"])
        return {"loss": s["loss"], "dlogits": s["dlogits"]}
    moe.moe_fp8_matmul(s["x8"], s["x_scale"], s["w"], s["w_scale"], s["y"], s["ws"], offsets=s["offsets"],
                       rows=s["rows"])
    return {"y": s["y"]}


def _norm(s):
    x, r = s["x"].float(), s["residual"].float()
    T, n = x.shape
    h = x + r
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    kb = -(-n // GROUP)
    pad = torch.zeros(T, kb * GROUP, device=x.device)
    pad[:, :n] = v
    pad = pad.reshape(T, kb, GROUP)
    amax = pad.abs().amax(2)
    scale = amax / FP8_MAX
    inv = torch.where(amax > 0, FP8_MAX / amax, torch.zeros_like(amax))
    x8 = (pad * inv[:, :, None]).reshape(T, kb * GROUP)[:, :n].to(torch.float8_e4m3fn)
    return {"residual": h.to(s["x"].dtype), "y": v.to(s["x"].dtype), "x8": x8, "scale": scale}


def _order(s):
    counts, offsets, rows, pos = _sorted(s["ids"], s["case"]["E"])
    return {"counts": counts, "offsets": offsets, "rows": rows, "pos": pos}


def _balance(s):
    l, E = s["logits"].float(), s["case"]["E"]
    if s["case"]["gating"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        slope = p
    else:
        g = 1.0 / (1.0 + torch.exp(-l))
        p = g / g.sum(1, keepdim=True)
        slope = p * (1.0 / (1.0 + torch.exp(l)))
    N = s["counts"].sum()
    f = (s["counts"] * E).float() / N
    coef = s["alpha"] * s["k"] / N.float()
    valid = s["valid"].float()[:, None]
    g = (p * f).sum(1, keepdim=True)
    some = N > 0
    loss = torch.where(some, coef * (g * valid).double().sum().float(), torch.zeros_like(coef)).reshape(1)
    grad = torch.where(some, s["grad_loss"] * coef * slope * (f - g) * valid, torch.zeros_like(l))
    return {"loss": loss, "dlogits": grad.to(s["logits"].dtype)}


def _matmul(s):
    x8, w, K = s["x8"], s["w"], s["x8"].shape[1]
    x = x8.float() * s["x_scale"].repeat_interleave(GROUP, 1)[:, :K]
    N = w.shape[-2]
    if s["rows"] is None:
        wf = w.float() * s["w_scale"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
        return {"y": (x @ wf.t()).to(s["y"].dtype)}
    E = w.shape[0]
    xs = torch.zeros(E, s["cap"], K, device=x.device)
    xs[s["group"], s["at"]] = x[s["rows"].long()]
    wf = w.float() * s["w_scale"].repeat_interleave(GROUP, 1)[:, :N].repeat_interleave(GROUP, 2)[:, :, :K]
    y = torch.bmm(xs, wf.transpose(1, 2))
    return {"y": y[s["group"], s["at"]].to(s["y"].dtype)}


# ------------------------------------------------------------------- work

def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        n, b = case["n"], BYTES[case["type"]]
        return {"bytes": T * n * (4 * b + 1) + T * -(-n // GROUP) * 4 + 4 * n, "flops": 10 * T * n}
    if op == "order":
        k, E = min(case["k"], case["E"]), case["E"]
        return {"bytes": 12 * T * k + 4 * (2 * E + 1), "flops": 0}
    if op == "balance":
        E = case["E"]
        return {"bytes": 2 * T * E * BYTES[case["type"]] + T + 4 * E, "flops": 12 * T * E}
    k, E, N, K = case["k"], case["E"], case["N"], case["K"]
    kb, nb = -(-K // GROUP), -(-N // GROUP)
    hit = 1 if E == 1 else E * (1 - (1 - k / E) ** T)     # experts that some token chose
    return {"bytes": T * (K + 4 * kb) + hit * (N * K + 4 * nb * kb) + T * k * N * BYTES[case["type"]],
            "flops": 2 * T * k * N * K}


# ------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        T, n = case["T"], case["n"]
        out = {"residual": torch.empty(T, n, dtype=torch.float64, device="cuda")}
        out["y"] = torch.empty_like(out["residual"])
        out["x8"] = torch.empty_like(out["residual"])      # before the rounding to 8 bits
        out["scale"] = torch.empty(T, -(-n // GROUP), dtype=torch.float64, device="cuda")
        out["residual"].copy_(s["x"]).add_(s["residual"])
        mean = torch.linalg.vector_norm(out["residual"], dim=1).square() / n
        torch.mul(out["residual"] / torch.sqrt(mean + EPS)[:, None], s["weight"], out=out["y"])
        for b in range(out["scale"].shape[1]):
            part = out["y"][:, b * GROUP:(b + 1) * GROUP]
            out["scale"][:, b] = part.abs().max(dim=1).values / FP8_MAX
            out["x8"][:, b * GROUP:(b + 1) * GROUP] = part / out["scale"][:, b:b + 1]
        return out
    if op == "order":
        return None     # whole numbers: nothing is rounded
    if op == "balance":
        l, E = s["logits"].double(), case["E"]
        live = s["valid"].bool()
        share = torch.log_softmax(l, 1) if case["gating"] == "softmax" else \
            torch.nn.functional.logsigmoid(l) - torch.logsumexp(torch.nn.functional.logsigmoid(l), 1, keepdim=True)
        p = torch.exp(share)
        c = s["counts"].double()
        N = float(c.sum())
        if not N:
            return {"loss": torch.zeros(1, dtype=torch.float64), "dlogits": torch.zeros_like(l)}
        factor = s["alpha"] * E * s["k"] / (N * N)
        dot = p @ c
        slope = p if case["gating"] == "softmax" else p * torch.sigmoid(-l)
        grad = s["grad_loss"].double() * factor * slope * (c[None, :] - dot[:, None])
        grad[~live] = 0
        return {"loss": (factor * dot[live].sum()).reshape(1), "dlogits": grad}
    k, E, N, K = case["k"], case["E"], case["N"], case["K"]
    if 2 * T_k(case) * N * K > 4e12:
        return {"y": None}
    wide = torch.arange(K, device="cuda") // GROUP
    tall = torch.arange(N, device="cuda") // GROUP
    x = s["x8"].double() * s["x_scale"].double()[:, wide]
    y = torch.zeros(T_k(case), N, dtype=torch.float64, device="cuda")
    w, ws = (s["w"][None], s["w_scale"][None]) if E == 1 else (s["w"], s["w_scale"])
    ends = [0, T_k(case)] if E == 1 else s["offsets"].tolist()
    for g in range(E):
        a, b = ends[g], ends[g + 1]
        if a < b:
            rows = slice(a, b) if E == 1 else s["rows"][a:b].long()
            y[a:b] = x[rows] @ (w[g].double() * ws[g].double()[tall][:, wide]).t()
    return {"y": y}


def T_k(case):
    return case["T"] * case["k"]
