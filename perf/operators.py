"""Cases of the routing and 8-bit integer operators, with their plain forms.

Four operators: the routing of tokens to experts (`route`), the product in 8-bit integers of rows
quantised on the way (`gemm`), the same product over the rows of each expert (`experts`) and the
gated sum of the experts' outputs (`combine`).  `own` chooses between the plain form, elementary
torch operations, and the framework's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token of the K3-shaped layer: softmax scores, latency only
        route("route_token", rows=1, experts=896, top_k=16),
        # a verify step's rows through a grouped router with a balance bias
        route("route_verify", rows=64, experts=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
              group_top=2, scale=2.5),
        # an odd chunk of a prompt, 16-bit logits, the best expert choosing its group, gates not renormalised; a padded tail
        route("route_chunk", rows=4093, experts=160, top_k=6, dtype="bf16", groups=8, top_groups=3, group_top=1,
              renorm=False, scale=16.0, pad=61),
        # a long prompt through a K3-sized router with a balance bias
        route("route_prompt", rows=16384, experts=896, top_k=16, score="sigmoid", bias=True),
        # one token through a square matrix of the dense trunk
        gemm("gemm_token", m=1, n=7168, k=7168),
        # a ragged decode batch through an expert-sized matrix
        gemm("gemm_rows", m=37, n=1536, k=7168, dtype="f32", out="f32"),
        # an odd chunk of a prompt through a shared expert's gate and up matrices
        gemm("gemm_chunk", m=509, n=1536, k=7168, dtype="f16", out="f16", swiglu=True),
        # a long prompt through a square matrix of the dense trunk
        gemm("gemm_prompt", m=8192, n=7168, k=7168),
        # a verify step's 8 rows through the gate and up matrices of 16 of 128 experts each: bound by the weights
        experts("experts_verify", tokens=8, experts=128, top_k=16, n=1024, k=7168, swiglu=True),
        # a prompt through the experts' down matrices, padded at its end: bound by the matrix units
        experts("experts_prompt", tokens=4096, experts=64, top_k=8, n=7168, k=1536, by_slot=True, pad=37),
        # one token's 16 expert outputs
        combine("combine_token", tokens=1, top_k=16, hidden=7168),
        # a prompt's expert outputs: bound by reading them
        combine("combine_prompt", tokens=4096, top_k=16, hidden=7168),
    ]


def route(name=None, rows=1, experts=64, top_k=4, dtype="f32", score="softmax", bias=False, groups=1, top_groups=1,
          group_top=1, renorm=True, scale=1.0, pad=0):
    return _case(name, op="route", rows=rows, experts=experts, top_k=top_k, dtype=dtype, score=score, bias=bias,
                 groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale, pad=pad)


def gemm(name=None, m=1, n=64, k=64, dtype="bf16", out="bf16", swiglu=False):
    return _case(name, op="gemm", m=m, n=n, k=k, dtype=dtype, out=out, swiglu=swiglu)


def experts(name=None, tokens=1, experts=8, top_k=2, n=64, k=64, dtype="bf16", out="bf16", swiglu=False, by_slot=False,
            pad=0):
    return _case(name, op="experts", tokens=tokens, experts=experts, top_k=top_k, n=n, k=k, dtype=dtype, out=out,
                 swiglu=swiglu, by_slot=by_slot, pad=pad)


def combine(name=None, tokens=1, top_k=2, hidden=64, dtype="bf16"):
    return _case(name, op="combine", tokens=tokens, top_k=top_k, hidden=hidden, dtype=dtype)


def _case(name, **values):
    return values if name is None else {"name": name, **values}


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    kind = rng.choice(["route", "gemm", "gemm", "experts", "combine"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _spread(rng, 8, 1024 // groups)
        top_groups = rng.randint(1, groups)
        rows = _spread(rng, 1, 16384 * 896 // max(896, groups * size))
        return route(rows=rows, experts=groups * size,
                     top_k=min(_spread(rng, 1, 32), top_groups * size), dtype=rng.choice(list(DTYPES)),
                     score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                     top_groups=top_groups, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                     scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, rows // 9]))
    if kind == "gemm":
        n, k, swiglu = _spread(rng, 64, 8192), 16 * _spread(rng, 4, 512), rng.random() < 0.3
        most = 8192 * 7168 * 7168 // (n * k * (2 if swiglu else 1))
        return gemm(m=_spread(rng, 1, min(8192, most)), n=n, k=k, dtype=rng.choice(list(DTYPES)),
                    out=rng.choice(list(DTYPES)), swiglu=swiglu)
    if kind == "experts":
        number, k, swiglu = _spread(rng, 2, 128), 16 * _spread(rng, 8, 448), rng.random() < 0.5
        n = _spread(rng, 64, min(7168, 128 * 2 * 1024 * 7168 // (number * k * (2 if swiglu else 1))))
        top_k = _spread(rng, 1, min(16, number))
        most = 4096 * 8 * 7168 * 1536 // (n * k * (2 if swiglu else 1) * top_k)
        tokens = _spread(rng, 1, max(1, min(4096, most)))
        return experts(tokens=tokens, experts=number, top_k=top_k, n=n, k=k, dtype=rng.choice(list(DTYPES)),
                       out=rng.choice(list(DTYPES)), swiglu=swiglu, by_slot=rng.random() < 0.5,
                       pad=rng.choice([0, tokens // 9]))
    return combine(tokens=_spread(rng, 1, 4096), top_k=_spread(rng, 1, 16), hidden=_spread(rng, 64, 7168),
                   dtype=rng.choice(["bf16", "f16"]))


# ---- inputs -------------------------------------------------------------------------------------------------------


def _codes(gen, *shape):
    """Weights as they come out of a per-channel quantisation: normal values, the largest of a channel near 127."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    for i in range(shape[0]):  # a matrix at a time: the fp32 numbers of all experts need not exist together
        v = torch.randn(shape[1:], generator=gen, device="cuda")
        out[i] = (v * 31.0).round_().clamp_(-127.0, 127.0).to(torch.int8)
    return out


def _rows(gen, rows, k, dtype):
    """Normalised activations, with a few channels that are larger than the others."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    loud = torch.rand(k, generator=gen, device="cuda") < 0.01
    return (x * torch.where(loud, 6.0, 1.0)).to(DTYPES[dtype])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "route":
        rows, number = case["rows"], case["experts"]
        logits = (torch.randn(rows, number, generator=gen, device="cuda") * 1.7).to(DTYPES[case["dtype"]])
        if case["pad"]:
            logits[rows - case["pad"]:] = -math.inf  # padded rows take no expert
        bias = torch.randn(number, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        return {"logits": logits, "bias": bias}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        parts = 2 if case["swiglu"] else 1
        return {"x": _rows(gen, m, k, case["dtype"]), "w": _codes(gen, parts, n, k),
                "w_scale": (torch.rand(parts, n, generator=gen, device="cuda") + 0.5) * (0.02 / 31.0)}
    if op == "experts":
        tokens, number, top_k, n, k = (case[a] for a in ("tokens", "experts", "top_k", "n", "k"))
        parts = 2 if case["swiglu"] else 1
        popular = torch.rand(number, generator=gen, device="cuda").mul_(1.5)  # some experts are chosen more often
        score = popular + torch.rand(tokens, number, generator=gen, device="cuda")
        idx = score.topk(top_k, dim=1).indices.to(torch.int32)
        if case["pad"]:
            idx[tokens - case["pad"]:] = -1
        rows = tokens * top_k if case["by_slot"] else tokens
        return {"x": _rows(gen, rows, k, case["dtype"]), "idx": idx, "w": _codes(gen, number, parts, n, k),
                "w_scale": (torch.rand(number, parts, n, generator=gen, device="cuda") + 0.5) * (0.02 / 31.0)}
    tokens, top_k, hidden = case["tokens"], case["top_k"], case["hidden"]
    gate = torch.rand(tokens, top_k, generator=gen, device="cuda") + 0.05
    return {"residual": torch.randn(tokens, hidden, generator=gen, device="cuda"), "gate": gate / gate.sum(1, keepdim=True),
            "y": torch.randn(tokens * top_k, hidden, generator=gen, device="cuda").to(DTYPES[case["dtype"]])}


def prepare(case, seed):
    state = {"case": dict(case), **_inputs(case, seed)}
    if not own:
        return state
    import memory_bound_mxfp4_amd as moe
    op = case["op"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    # a serving program keeps its output buffers and workspaces
    if op == "route":
        state["topk"] = (empty((case["rows"], case["top_k"]), torch.int32), empty((case["rows"], case["top_k"]), torch.float32))
    elif op == "gemm":
        state["out"] = empty((case["m"], case["n"]), DTYPES[case["out"]])
        state["ws"] = empty((moe.gemm_i8_workspace_size(case["m"], case["n"], case["k"], case["swiglu"], state["x"].dtype),),
                            torch.uint8)
    elif op == "experts":
        slots = case["tokens"] * case["top_k"]
        state["out"] = empty((slots, case["n"]), DTYPES[case["out"]])
        state["groups"] = moe.alloc_slot_groups(case["tokens"], case["top_k"], case["experts"], device="cuda")
        size = moe.experts_gemm_i8_workspace_size(state["groups"], state["x"].shape[0], case["n"], case["k"], case["swiglu"],
                                                  state["x"].dtype)
        state["ws"] = empty((size,), torch.uint8)
    else:
        state["out"] = empty((case["tokens"], case["hidden"]), torch.float32)
    return state


# ---- one pass -----------------------------------------------------------------------------------------------------


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import memory_bound_mxfp4_amd as moe
        if op == "route":
            idx, gate = moe.moe_route(state["logits"], case["top_k"], bias=state["bias"], score=case["score"],
                                      groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                                      renorm=case["renorm"], scale=case["scale"], idx=state["topk"][0], gate=state["topk"][1])
            return {"idx": idx, "gate": gate}
        if op == "gemm":
            w, w_scale = (state["w"], state["w_scale"]) if case["swiglu"] else (state["w"][0], state["w_scale"][0])
            return moe.gemm_i8(state["x"], w, w_scale, swiglu=case["swiglu"], out=state["out"], ws=state["ws"])
        if op == "experts":
            groups = moe.moe_group_slots(state["idx"], case["experts"], groups=state["groups"])
            w, w_scale = (state["w"], state["w_scale"]) if case["swiglu"] else (state["w"][:, 0], state["w_scale"][:, 0])
            y = moe.experts_gemm_i8(state["x"], groups, w, w_scale, swiglu=case["swiglu"], out=state["out"], ws=state["ws"])
            return {"order": groups.order, "offsets": groups.offsets, "y": y}
        return moe.moe_combine(state["y"], state["gate"], residual=state["residual"], out=state["out"])
    if op == "route":
        return _plain_route(state, case)
    if op == "gemm":
        q, scale = _plain_quant(state["x"])
        return _plain_product(q, scale, state["w"], state["w_scale"]).to(DTYPES[case["out"]])
    if op == "experts":
        return _plain_experts(state, case)
    tokens, top_k, hidden = case["tokens"], case["top_k"], case["hidden"]
    y = state["y"].float().view(tokens, top_k, hidden)
    return state["residual"] + (y * state["gate"][:, :, None]).sum(1)


def _plain_route(state, case):
    """Scores and keys in 64 bits: two experts whose keys differ past the 32nd bit have an order all the same."""
    number, groups, top_k = case["experts"], case["groups"], case["top_k"]
    logits = state["logits"].float()
    valid = ~torch.isnan(logits) & (logits != -math.inf)
    lg = logits.clamp(max=torch.finfo(torch.float32).max).double().masked_fill(~valid, -math.inf)
    if case["score"] == "softmax":
        top = lg.amax(1, keepdim=True).clamp(min=-torch.finfo(torch.float32).max)
        e = torch.exp(lg - top)
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-lg))
    total = score if state["bias"] is None else score + state["bias"].double()
    total = total.masked_fill(~valid, -math.inf)
    key = lg if state["bias"] is None else total
    if groups > 1:
        best = total.view(-1, groups, number // groups).sort(dim=2, descending=True).values[:, :, :case["group_top"]]
        any_valid = best[:, :, 0] > -math.inf
        worth = torch.where(torch.isinf(best), 0.0, best).sum(2).masked_fill(~any_valid, -math.inf)
        rank = worth.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, rank, True)
        key = key.masked_fill(~kept.repeat_interleave(number // groups, dim=1), -math.inf)
    order = key.sort(dim=1, descending=True, stable=True)
    idx, found = order.indices[:, :top_k], order.values[:, :top_k] > -math.inf
    gate = score.gather(1, idx).masked_fill(~found, 0.0)
    if case["renorm"]:
        total = gate.sum(1, keepdim=True)
        gate = torch.where(total > 0, gate / total, 0.0)
    return {"idx": idx.masked_fill(~found, -1).to(torch.int32), "gate": (gate * case["scale"]).float()}


def _plain_quant(x):
    """Rows to 8 bits. The quotient is taken in 64 bits: next to the middle between two codes 32 decide wrongly."""
    v = x.double()
    scale = (v.abs().amax(1) / 127.0).float()
    q = torch.where(scale[:, None] > 0, torch.round(v / scale.double()[:, None]), 0.0).clamp(-127.0, 127.0)
    return q.float(), scale


def _plain_product(q, scale, w, w_scale):
    """q [rows][k] with the one or two matrices of w [parts][n][k]; two are a gate and an up matrix."""
    y = [(q @ w[p].float().t()) * scale[:, None] * w_scale[p][None, :] for p in range(w.shape[0])]
    return y[0] if len(y) == 1 else y[0] / (1.0 + torch.exp(-y[0])) * y[1]


def _plain_experts(state, case):
    number, top_k = case["experts"], case["top_k"]
    flat = state["idx"].reshape(-1).long()
    flat = torch.where(flat < 0, number, flat)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(number + 1, device=flat.device)[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    q, scale = _plain_quant(state["x"])
    y = torch.zeros(flat.numel(), case["n"], dtype=DTYPES[case["out"]], device=flat.device)
    ends = offsets.tolist()
    for e in range(number):
        if ends[e + 1] > ends[e]:
            slots = order[ends[e]:ends[e + 1]]
            rows = slots if case["by_slot"] else slots // top_k
            y[slots] = _plain_product(q[rows], scale[rows], state["w"][e], state["w_scale"][e]).to(y.dtype)
    return {"order": order.to(torch.int32), "offsets": offsets.to(torch.int32), "y": y}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "route":
        rows, number = case["rows"], case["experts"]
        return {"bytes": rows * number * BYTES[case["dtype"]] + (4 * number if case["bias"] else 0) + rows * case["top_k"] * 8,
                "flops": 4 * rows * number}
    if op == "gemm":
        m, n, k, parts = case["m"], case["n"], case["k"], 2 if case["swiglu"] else 1
        return {"bytes": m * k * BYTES[case["dtype"]] + parts * n * (k + 4) + m * n * BYTES[case["out"]],
                "flops": 2 * m * n * k * parts}
    if op == "experts":
        tokens, number, top_k, n, k = (case[a] for a in ("tokens", "experts", "top_k", "n", "k"))
        parts, real = 2 if case["swiglu"] else 1, tokens - case["pad"]
        used = number * (1.0 - (1.0 - top_k / number) ** real)  # experts that some token is expected to take
        return {"bytes": round(real * (top_k if case["by_slot"] else 1) * k * BYTES[case["dtype"]] + used * parts * n * (k + 4)
                               + tokens * top_k * (n * BYTES[case["out"]] + 8) + 4 * number),
                "flops": 2 * real * top_k * n * k * parts}
    tokens, top_k, hidden = case["tokens"], case["top_k"], case["hidden"]
    return {"bytes": tokens * top_k * (hidden * BYTES[case["dtype"]] + 4) + 8 * tokens * hidden,
            "flops": 2 * tokens * top_k * hidden}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------


def exact(case, seed):
    data = _inputs(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(data, case)
    if op == "gemm":
        return _exact_product(data["x"], data["w"], data["w_scale"])
    if op == "experts":
        tokens, top_k, number = case["tokens"], case["top_k"], case["experts"]
        where = data["idx"].reshape(-1)
        y = torch.zeros(tokens * top_k, case["n"], dtype=torch.float64, device="cuda")
        order, ends = [], [0]
        for e in range(number):
            slots = torch.nonzero(where == e).flatten()
            order.append(slots)
            ends.append(ends[-1] + slots.numel())
            if slots.numel():
                x = data["x"][slots] if case["by_slot"] else data["x"][torch.div(slots, top_k, rounding_mode="floor")]
                y[slots] = _exact_product(x, data["w"][e], data["w_scale"][e])
        order.append(torch.nonzero((where < 0) | (where >= number)).flatten())
        ends.append(tokens * top_k)
        return {"order": torch.cat(order).to(torch.int32), "offsets": torch.tensor(ends, dtype=torch.int32, device="cuda"), "y": y}
    out = data["residual"].double()
    y = data["y"].view(case["tokens"], case["top_k"], case["hidden"])
    for j in range(case["top_k"]):
        out += data["gate"][:, j].double()[:, None] * y[:, j].double()
    return out


def _exact_product(x, w, w_scale):
    wide = x.to(torch.float64)
    step = torch.div(wide.abs().max(dim=1, keepdim=True).values, 127.0).to(torch.float32).to(torch.float64)
    codes = torch.where(step > 0, wide / torch.where(step > 0, step, 1.0), torch.zeros_like(wide)).round().clamp(-127, 127)
    parts = []
    for p in range(w.shape[0]):
        total = torch.matmul(codes, w[p].to(torch.float64).transpose(0, 1).contiguous())
        parts.append(total * (step * w_scale[p].to(torch.float64)))
    if len(parts) == 1:
        return parts[0]
    return parts[1] * (parts[0] * torch.sigmoid(parts[0]))


def _exact_route(data, case):
    """The best expert, top_k times over, in place of a sort."""
    number, groups = case["experts"], case["groups"]
    values = data["logits"].to(torch.float64)
    usable = torch.logical_not(torch.isnan(values) | torch.isneginf(values))
    values = torch.where(usable, values.clamp(max=torch.finfo(torch.float32).max), torch.full_like(values, -math.inf))
    if case["score"] == "softmax":
        score = torch.softmax(values, dim=1)
    else:
        score = torch.sigmoid(values)
    score = torch.where(usable, score, torch.zeros_like(score))
    ranked = score if data["bias"] is None else score + data["bias"].to(torch.float64)
    places = torch.arange(number, device="cuda")
    allowed = usable.clone()
    if groups > 1:
        inside = torch.where(usable, ranked, torch.full_like(ranked, -math.inf)).view(-1, groups, number // groups)
        worth = torch.zeros(inside.shape[:2], dtype=torch.float64, device="cuda")
        left = inside.clone()
        for _ in range(min(case["group_top"], number // groups)):
            best, at = left.max(dim=2, keepdim=True)
            worth += torch.where(torch.isneginf(best), torch.zeros_like(best), best)[:, :, 0]
            left.scatter_(2, at, -math.inf)
        open_groups = usable.view(-1, groups, number // groups).any(2)
        worth = torch.where(open_groups, worth, torch.full_like(worth, -math.inf))
        names = torch.arange(groups, device="cuda")
        kept = torch.zeros_like(open_groups)
        for _ in range(case["top_groups"]):
            best = worth.max(1, keepdim=True).values
            first = torch.where((worth == best) & ~kept, names, groups).min(1, keepdim=True).values
            chosen = (names == first) & torch.logical_not(torch.isneginf(best))
            kept |= chosen
            worth = torch.where(chosen, torch.full_like(worth, -math.inf), worth)
        allowed &= kept.repeat_interleave(number // groups, dim=1)
    key = torch.where(allowed, values if data["bias"] is None else ranked, torch.full_like(ranked, -math.inf))
    idx, gate = [], []
    for _ in range(case["top_k"]):
        best = key.max(1, keepdim=True).values
        some = torch.logical_not(torch.isneginf(best))
        first = torch.where(key == best, places, number).min(1, keepdim=True).values
        idx.append(torch.where(some, first, -1))
        gate.append(torch.where(some, score.gather(1, first.clamp(max=number - 1)), 0.0))
        key = torch.where(places == first, torch.full_like(key, -math.inf), key)
    idx, gate = torch.cat(idx, 1), torch.cat(gate, 1)
    if case["renorm"]:
        whole = gate.sum(1, keepdim=True)
        gate = torch.where(whole > 0, gate / whole, torch.zeros_like(gate))
    return {"idx": idx.to(torch.int32), "gate": gate * case["scale"]}
