"""The operators of a layer of experts with 4-bit weights, as they are measured.

A router (scores, a bias for balance, groups of experts, the best few, their weights) and its gradient, the grouping of
routes by expert, the product with 4-bit weights that have a scale for each group of k, and the same product (plain or
gated) over routes that are grouped by expert.  ``run`` computes each in plain torch operations, or, where ``own`` is
true, by the package's own calls.

Activations are int8 with one scale a token, four to an int32 word as everywhere in the package.  4-bit weights are two's
complement, eight to an int32 word: of each 16 bytes (32 neighbours of k) byte b holds element b in its low four bits and
element 16 + b in its high four.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def listed():
    return [
        # One decoded token through the router of a wide layer of experts (grouped, balanced by a bias): latency.
        {"name": "route_one_token", "op": "route", "tokens": 1, "experts": 256, "dtype": "float32", "top_k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True},
        # An odd batch over a count of experts that is no power of two, half-precision logits with many ties.
        {"name": "route_odd_batch", "op": "route", "tokens": 1003, "experts": 60, "dtype": "bfloat16", "top_k": 4,
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renormalize": False},
        # A long prompt (or a training batch) through the same router as the first.
        {"name": "route_prompt", "op": "route", "tokens": 65536, "experts": 256, "dtype": "float32", "top_k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True},
        # The router's gradient for a small batch, renormalised weights.
        {"name": "route_backward_small", "op": "route_backward", "tokens": 187, "experts": 64, "dtype": "float32",
         "top_k": 6, "score": "softmax", "renormalize": True},
        # The router's gradient for a training batch: every logit takes part through the softmax's sum.
        {"name": "route_backward_batch", "op": "route_backward", "tokens": 65536, "experts": 256, "dtype": "bfloat16",
         "top_k": 8, "score": "softmax", "renormalize": False},
        # The routes of a decode batch grouped by expert: latency.
        {"name": "group_decode", "op": "group", "tokens": 64, "routes": 8, "experts": 256},
        # The routes of a training batch.
        {"name": "group_prompt", "op": "group", "tokens": 65536, "routes": 8, "experts": 256},
        # A projection for one decoded token: the 4-bit weights are read once.
        {"name": "i4_one_token", "op": "matmul", "tokens": 1, "rows": 16384, "k": 8192, "group": 128, "dtype": "bfloat16",
         "scales": "float16", "bias": False},
        # A small decode batch, ragged everywhere, with the smallest groups and a bias.
        {"name": "i4_ragged_batch", "op": "matmul", "tokens": 21, "rows": 4099, "k": 11008, "group": 32, "dtype": "float16",
         "scales": "bfloat16", "bias": True},
        # A prompt through the down projection: matrix-core rate.
        {"name": "i4_prompt", "op": "matmul", "tokens": 4096, "rows": 8192, "k": 28672, "group": 128, "dtype": "bfloat16",
         "scales": "float16", "bias": False},
        # A decode batch through the experts' gated projections: nearly every expert's weights are read for a few rows.
        {"name": "experts_gated_decode", "op": "experts", "tokens": 32, "routes": 8, "experts": 128, "rows": 2048, "k": 4096,
         "group": 128, "dtype": "float32", "scales": "float16", "act": "silu", "missing": False},
        # A prompt through the experts' down projections, each route a row of its own.
        {"name": "experts_down_prompt", "op": "experts", "tokens": 4096, "routes": 8, "experts": 64, "rows": 4096, "k": 2048,
         "group": 128, "dtype": "float32", "scales": "float16", "act": None, "missing": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_backward", "group", "matmul", "experts"))
    tokens = _log(rng, 1, 65536)
    if op in ("route", "route_backward", "group"):
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * _log(rng, max(1, 4 // groups), 256 // groups)
        top_k = rng.randint(1, min(8, experts))
        if op == "group":
            return {"op": op, "tokens": tokens, "routes": top_k, "experts": experts}
        case = {"op": op, "tokens": tokens, "experts": experts, "dtype": rng.choice(sorted(DTYPES)), "top_k": top_k,
                "score": rng.choice(("softmax", "sigmoid")), "renormalize": rng.random() < 0.5}
        if op == "route_backward":
            return case
        top_groups = rng.randint(1, groups)
        while top_groups * (experts // groups) < top_k:
            top_groups += 1
        case.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)))
        return case
    group = rng.choice((32, 64, 128, 256))
    # row lengths: any multiple of 32, or, as most layers have them, of 256
    k = 32 * _log(rng, 2, 512) if rng.random() < 0.5 else 256 * _log(rng, 1, 64)
    rows = _log(rng, 32, 28672)
    case = {"op": op, "rows": rows, "k": k, "group": group, "dtype": rng.choice(sorted(DTYPES)),
            "scales": rng.choice(sorted(DTYPES))}
    # no dearer than the largest listed case of the operator
    if op == "matmul":
        case["tokens"] = max(1, min(_log(rng, 1, 8192), 4096 * 8192 * 28672 // (rows * k)))
        case["bias"] = rng.random() < 0.5
        return case
    case["experts"] = max(1, min(_log(rng, 2, 256), 128 * 2 * 2048 * 4096 // (2 * rows * k)))
    case["routes"] = rng.randint(1, min(8, case["experts"]))
    case["tokens"] = max(1, min(_log(rng, 1, 8192), 4096 * 8 * 4096 * 2048 // (2 * rows * k * case["routes"])))
    case["act"] = rng.choice((None,) + ACTS)
    case["missing"] = rng.random() < 0.3
    return case


# ------------------------------------------------------------------ inputs

def _pack4(q):
    """int8 values -8 .. 7 [..., k] -> packed int32 [..., k / 8]."""
    b = q.view(torch.uint8).reshape(*q.shape[:-1], q.shape[-1] // 32, 2, 16)
    return ((b[..., 0, :] & 15) | (b[..., 1, :] << 4)).reshape(*q.shape[:-1], q.shape[-1] // 2).view(torch.int32)


def _weights(experts, rows, k, group, scales, g):
    """Normally distributed weights of 1/sqrt(k), rounded to 4 bits with one scale for each group of k."""
    parts, most = [], max(1, 2 ** 28 // (rows * k))
    for e in range(0, experts, most):
        n = min(most, experts - e)
        q = torch.randn(n, rows, k, generator=g, device="cuda").mul_(2.5).round_().clamp_(-8, 7).to(torch.int8)
        parts.append(_pack4(q))
    scale = (0.5 + torch.rand(experts, rows, -(-k // group), generator=g, device="cuda")) / (2.5 * math.sqrt(k))
    return parts[0] if len(parts) == 1 else torch.cat(parts), scale.to(DTYPES[scales])


def _activations(tokens, k, g):
    """Hidden states with a few channels that are much larger than the rest, quantised by token."""
    x = torch.randn(tokens, k, generator=g, device="cuda", dtype=torch.float32)
    x *= 1.0 + 4.0 * (torch.rand(k, generator=g, device="cuda") < 0.005)
    scale = x.abs().amax(1) / 127.0
    q = (x / scale[:, None]).round_().clamp_(-127, 127).to(torch.int8)
    return q.view(torch.int32), scale


def _logits(tokens, experts, g):
    """Router logits: some experts are more popular than others."""
    return 1.5 * torch.randn(tokens, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    tokens = case["tokens"]
    if case["op"] in ("route", "route_backward"):
        s["logits"] = _logits(tokens, case["experts"], g).to(DTYPES[case["dtype"]])
        if case["op"] == "route":
            s["bias"] = 0.05 * torch.randn(case["experts"], generator=g, device="cuda") if case["bias"] else None
        else:
            s["ids"] = torch.topk(s["logits"].float(), case["top_k"], dim=1).indices.to(torch.int32)
            s["d_weights"] = torch.randn(tokens, case["top_k"], generator=g, device="cuda")
        return s
    if case["op"] == "group":
        s["ids"] = torch.topk(_logits(tokens, case["experts"], g), case["routes"], dim=1).indices.to(torch.int32)
        # a few routes lead to experts that another device holds
        s["ids"][torch.rand(tokens, case["routes"], generator=g, device="cuda") < 0.02] = -1
        return s
    rows, k, group = case["rows"], case["k"], case["group"]
    if case["op"] == "matmul":
        s["x"], s["x_scale"] = _activations(tokens, k, g)
        w, scale = _weights(1, rows, k, group, case["scales"], g)
        s["w"], s["w_scale"] = w[0], scale[0]
        s["bias"] = torch.randn(rows, generator=g, device="cuda") if case["bias"] else None
        return s
    experts, routes = case["experts"], case["routes"]
    s["w"], s["w_scale"] = _weights(experts, rows, k, group, case["scales"], g)
    ids = torch.topk(_logits(tokens, experts, g), routes, dim=1).indices.to(torch.int32)
    if case["missing"]:
        ids[torch.rand(tokens, routes, generator=g, device="cuda") < 0.3] = -1
    _, s["index"], s["offsets"] = _group(ids, experts)
    if case["act"] is not None:
        # the gated projection reads each token's row for all of its routes
        s["w_up"], s["up_scale"] = _weights(experts, rows, k, group, case["scales"], g)
        s["x"], s["x_scale"] = _activations(tokens, k, g)
    else:
        s["x"], s["x_scale"] = _activations(tokens * routes, k, g)
        s["index"] = None
    # rows behind the last route that is held here stay as they are
    s["out"] = torch.zeros(tokens * routes, rows, dtype=DTYPES[case["dtype"]], device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "relu":
        return torch.where(g < 0, torch.zeros_like(g), g)
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _route(s):
    """Choices in 64 bits (neighbouring scores differ by less than a step of 32), weights in 32."""
    logits = s["logits"].double()
    top = logits.amax(1, keepdim=True)
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        e = torch.exp(logits - top)
        score = e / e.sum(1, keepdim=True)
    # without a bias the logits order the experts
    choice = logits if s["bias"] is None else score + s["bias"].double()
    tokens, experts = logits.shape
    if s["groups"] > 1:
        size = experts // s["groups"]
        ranked = (choice if s["group_top"] == 1 else score if s["bias"] is None else choice).view(tokens, s["groups"], size)
        best = torch.sort(ranked, dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros(tokens, s["groups"], dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(size, 1), choice, torch.full_like(choice, -math.inf))
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    weights = torch.gather(score, 1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return ids.to(torch.int32), (weights * 2.5).float()


def _route_backward(s):
    logits, ids, d = s["logits"].float(), s["ids"].long(), s["d_weights"] * 2.5
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    chosen = torch.gather(score, 1, ids)
    if s["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        d = (d - (d * chosen).sum(1, keepdim=True) / total) / total
    d_score = torch.zeros_like(score).scatter_add_(1, ids, d)
    if s["score"] == "sigmoid":
        out = d_score * score * (1 - score)
    else:
        out = score * (d_score - (d_score * score).sum(1, keepdim=True))
    return out.to(s["logits"].dtype)


def _group(ids, experts):
    """Routes in order of their experts: where each went, whose token each grouped row is, where each expert's begin."""
    tokens, routes = ids.shape
    flat = ids.reshape(-1).long()
    here = (flat >= 0) & (flat < experts)
    key = torch.where(here, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device="cuda")
    slots = torch.where(here, place, torch.full_like(place, -1)).to(torch.int32).view(tokens, routes)
    count = torch.zeros(experts + 1, dtype=torch.long, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(count[:experts], 0)
    rows = torch.where(key[order] < experts, order // routes, torch.full_like(order, -1))
    return slots, rows.to(torch.int32), offsets.to(torch.int32)


def _values4(w):
    """Packed 4-bit weights [..., k / 8] as f32 [..., k]."""
    b = w.view(torch.int8).reshape(*w.shape[:-1], w.shape[-1] // 4, 16)
    return torch.cat(((b << 4) >> 4, b >> 4), -1).reshape(*w.shape[:-1], w.shape[-1] * 8).float()


def _dense(w, scale, group):
    """Dequantised weights [rows][k] in f32."""
    return _values4(w) * scale.float().repeat_interleave(group, 1)[:, :w.shape[-1] * 8]


def _run_plain(s):
    op = s["op"]
    if op == "route":
        return _route(s)
    if op == "route_backward":
        return _route_backward(s)
    if op == "group":
        return _group(s["ids"], s["experts"])
    dtype = DTYPES[s["dtype"]]
    if op == "matmul":
        y = (s["x"].view(torch.int8).float() @ _dense(s["w"], s["w_scale"], s["group"]).t()) * s["x_scale"][:, None]
        return (y if s["bias"] is None else y + s["bias"]).to(dtype)
    out = torch.zeros_like(s["out"])
    bounds = s["offsets"].tolist()
    for e in range(s["experts"]):
        begin, end = bounds[e], bounds[e + 1]
        if begin == end:
            continue
        at = slice(begin, end) if s["index"] is None else s["index"][begin:end].long()
        x, xs = s["x"][at].view(torch.int8).float(), s["x_scale"][at][:, None]
        y = (x @ _dense(s["w"][e], s["w_scale"][e], s["group"]).t()) * xs
        if s["act"] is not None:
            y = _act(y, s["act"]) * ((x @ _dense(s["w_up"][e], s["up_scale"][e], s["group"]).t()) * xs)
        out[begin:end] = y.to(dtype)
    return out


def _run_own(s):
    import int8_dequant_dot_amd as loom

    op = s["op"]
    if op == "route":
        return loom.route_experts(s["logits"], s["top_k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                                  top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renormalize"],
                                  scale=2.5)
    if op == "route_backward":
        return loom.route_experts_backward(s["logits"], s["ids"], s["d_weights"], score=s["score"],
                                           renormalize=s["renormalize"], scale=2.5)
    if op == "group":
        return loom.group_routes(s["ids"], s["experts"])
    if op == "matmul":
        return loom.i4_matmul(s["w"], s["w_scale"], s["x"], s["x_scale"], bias=s["bias"], group=s["group"],
                              dtype=DTYPES[s["dtype"]])
    if s["act"] is None:
        return loom.i4_expert_matmul(s["w"], s["w_scale"], s["x"], s["x_scale"], s["offsets"], index=s["index"],
                                     group=s["group"], out=s["out"])
    return loom.i4_expert_gated_projection(s["w"], s["w_scale"], s["w_up"], s["up_scale"], s["x"], s["x_scale"],
                                           s["offsets"], index=s["index"], act=s["act"], group=s["group"], out=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the work and the 64-bit values

def work(case):
    op, t = case["op"], case["tokens"]
    size = {"float32": 4}.get(case.get("dtype"), 2)
    if op == "route":
        return {"bytes": t * case["experts"] * size + 8 * t * case["top_k"] + (4 * case["experts"] if case["bias"] else 0),
                "flops": 8 * t * case["experts"]}
    if op == "route_backward":
        e, k = case["experts"], case["top_k"]
        # the renormalised weights of the chosen, and sigmoids, need the chosen logits alone
        read = t * e if case["score"] == "softmax" and not case["renormalize"] else t * k
        return {"bytes": read * size + t * e * size + 8 * t * k, "flops": 8 * read}
    if op == "group":
        pairs = t * case["routes"]
        return {"bytes": 12 * pairs + 4 * (case["experts"] + 1), "flops": 2 * pairs}
    rows, k, groups = case["rows"], case["k"], -(-case["k"] // case["group"])
    weights = rows * k // 2 + rows * groups * {"float32": 4}.get(case["scales"], 2)
    if op == "matmul":
        return {"bytes": weights + t * (k + 4) + t * rows * size + (4 * rows if case["bias"] else 0), "flops": 2 * t * rows * k}
    pairs, matrices = t * case["routes"], 1 if case["act"] is None else 2
    x_rows = pairs if case["act"] is None else t
    # at most as many experts as routes are read
    read = min(case["experts"], pairs) * matrices * weights
    return {"bytes": read + x_rows * (k + 4) + pairs * (4 + rows * size), "flops": 2 * matrices * pairs * rows * k}


def _nibbles(w):
    """Packed weights as float64 [..., k], by arithmetic on unsigned bytes."""
    b = w.view(torch.uint8).to(torch.int16).unflatten(-1, (w.shape[-1] // 4, 16))
    n = torch.stack((b % 16, b // 16), -2).flatten(-3)
    return torch.where(n > 7, n - 16, n).double()


def _product64(x, w, scale, group):
    q = _nibbles(w)
    q *= scale.double()[:, torch.arange(q.shape[1], device="cuda") // group]
    return torch.mm(x, q.t().contiguous())


def _act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "relu":
        return g.clamp(min=0)
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2))
    # tanh z = 2 sigmoid(2 z) - 1, so the factor (1 + tanh z) / 2 is sigmoid(2 z)
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def _exact_route(s):
    l = s["logits"].double()
    t, e = l.shape
    score = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
    biased = s["bias"] is not None
    value = score + s["bias"].double() if biased else l
    open_ = torch.ones(t, s["groups"], dtype=torch.bool, device="cuda")
    if s["groups"] > 1:
        parts = (value if biased or s["group_top"] == 1 else score).unflatten(1, (s["groups"], -1))
        rank = torch.topk(parts, min(s["group_top"], parts.shape[2]), dim=2).values.sum(2)
        # a group stays if fewer than top_groups are better (greater, or equal and before it)
        before = torch.arange(s["groups"], device="cuda")
        better = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & (before[None, :] < before[:, None]))
        open_ = better.sum(2) < s["top_groups"]
    value = value.masked_fill(~open_.repeat_interleave(e // s["groups"], 1), -math.inf)
    ids = torch.empty(t, s["top_k"], dtype=torch.long, device="cuda")
    line = torch.arange(e, device="cuda").expand(t, e)
    for i in range(s["top_k"]):
        peak = value.amax(1, keepdim=True)
        ids[:, i] = torch.where(value == peak, line, e).amin(1)
        value = value.scatter(1, ids[:, i:i + 1], -math.inf)
    weights = torch.gather(score, 1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return ids.to(torch.int32), 2.5 * weights


def exact(case, seed):
    """The definitions in float64; grouped routes, which are whole numbers, by counting."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        with torch.enable_grad():
            l = s["logits"].double().requires_grad_()
            score = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
            w = torch.gather(score, 1, s["ids"].long())
            if s["renormalize"]:
                w = w / w.sum(1, keepdim=True)
            (2.5 * w * s["d_weights"].double()).sum().backward()
        return l.grad
    if op == "group":
        ids = s["ids"].reshape(-1).cpu().numpy()
        import numpy as np
        slots, rows = np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
        offsets = np.zeros(case["experts"] + 1, np.int32)
        at = 0
        for e in range(case["experts"]):
            mine = np.flatnonzero(ids == e)
            slots[mine] = np.arange(at, at + mine.size)
            rows[at:at + mine.size] = mine // case["routes"]
            at += mine.size
            offsets[e + 1] = at
        return tuple(torch.from_numpy(a).cuda() for a in (slots.reshape(case["tokens"], -1), rows, offsets))
    x = s["x"].view(torch.int8).double() * s["x_scale"].double()[:, None]
    if op == "matmul":
        y = _product64(x, s["w"], s["w_scale"], s["group"])
        return y if s["bias"] is None else y + s["bias"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for e, end in enumerate(s["offsets"][1:].tolist()):
        if end > begin:
            xe = x[begin:end] if s["index"] is None else x[s["index"][begin:end].long()]
            y = _product64(xe, s["w"][e], s["w_scale"][e], s["group"])
            if s["act"] is not None:
                y = _act64(y, s["act"]) * _product64(xe, s["w_up"][e], s["up_scale"][e], s["group"])
            out[begin:end] = y
        begin = end
    return out
