"""The int8 feed-forward operators, as they are measured.

Four operators on packed int8 data: a row quantiser (one scale a token), the int8 matrix product with a scale for each
token and each channel, the gated projection (both products, the activation and the product of the two), and that
projection's gradients.  ``run`` computes each in plain torch operations, or, where ``own`` is true, by the package's
own calls.  Weights are int8 with one scale a channel, activations int8 with one scale a token, both packed four to an
int32 word as everywhere in the package.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")
TINY = 2.0 ** -119  # a row whose largest magnitude is smaller quantises to zeros, scale 0


def listed():
    return [
        # The activations of one decoded token, quantised between two projections: launch latency.
        {"name": "quantize_one_token", "op": "quantize", "tokens": 1, "k": 8192, "dtype": "bfloat16"},
        # A long prompt's hidden activations, before the down projection: one large stream.
        {"name": "quantize_prompt", "op": "quantize", "tokens": 8191, "k": 28672, "dtype": "bfloat16"},
        # A projection for one decoded token: the weights are read once.
        {"name": "matmul_one_token", "op": "matmul", "tokens": 1, "rows": 16384, "k": 8192, "dtype": "bfloat16", "bias": False},
        # A small decode batch, ragged everywhere (a row count that is no tile's, an odd batch), with a bias.
        {"name": "matmul_ragged_batch", "op": "matmul", "tokens": 21, "rows": 4099, "k": 11008, "dtype": "float16", "bias": True},
        # A decode batch of 64 through a wide projection, logits-like f32 outputs.
        {"name": "matmul_64_tokens", "op": "matmul", "tokens": 64, "rows": 28672, "k": 8192, "dtype": "float32", "bias": False},
        # A prompt through the down projection: matrix-core rate.
        {"name": "matmul_prompt", "op": "matmul", "tokens": 4096, "rows": 8192, "k": 28672, "dtype": "bfloat16", "bias": False},
        # The gated projection of one decoded token.
        {"name": "gated_one_token", "op": "gated", "tokens": 1, "rows": 28672, "k": 8192, "dtype": "bfloat16", "act": "silu"},
        # A mid-sized batch (a chunk of a prompt beside decoding requests), odd, f32 out.
        {"name": "gated_chunk", "op": "gated", "tokens": 187, "rows": 11008, "k": 4096, "dtype": "float32", "act": "gelu_tanh"},
        # A prompt through the gated projection.
        {"name": "gated_prompt", "op": "gated", "tokens": 4096, "rows": 28672, "k": 8192, "dtype": "bfloat16", "act": "silu"},
        # Tuning over frozen int8 weights: a few tokens, f32 gradients.
        {"name": "backward_few_tokens", "op": "backward", "tokens": 5, "rows": 11008, "k": 4096, "dtype": "float32", "act": "silu"},
        # An ordinary micro-batch of odd length.
        {"name": "backward_micro_batch", "op": "backward", "tokens": 1003, "rows": 11008, "k": 4096, "dtype": "bfloat16", "act": "silu"},
        # A full training batch on the wide layer.
        {"name": "backward_batch", "op": "backward", "tokens": 2048, "rows": 28672, "k": 8192, "dtype": "bfloat16", "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "gated", "backward"))
    dtype = rng.choice(sorted(DTYPES))
    tokens = _log(rng, 1, 8192)
    # row lengths: any multiple of 4, or, as most layers have them, of 256
    k = 4 * _log(rng, 16, 4096) if rng.random() < 0.5 else 256 * _log(rng, 1, 64)
    case = {"op": op, "tokens": tokens, "k": k, "dtype": dtype}
    if op == "quantize":
        return case
    rows = _log(rng, 32, 28672)
    # no dearer than the largest listed case of the operator
    most = {"matmul": 4096 * 8192 * 28672, "gated": 4096 * 28672 * 8192, "backward": 2048 * 28672 * 8192}[op]
    case["tokens"] = max(1, min(tokens, most // (rows * k)))
    case["rows"] = rows
    if op == "matmul":
        case["bias"] = rng.random() < 0.5
    else:
        case["act"] = rng.choice(ACTS)
    return case


def _packed(t):
    return t.view(torch.int32)


def _weights(rows, k, g):
    """Normally distributed weights of 1/sqrt(k), rounded to int8 with one scale a row."""
    w = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.float32)
    q = w.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)
    scale = (0.5 + torch.rand(rows, generator=g, device="cuda")) / (32.0 * math.sqrt(k))
    return _packed(q), scale


def _activations(tokens, k, g):
    """Hidden states with a few channels that are much larger than the rest, quantised by token."""
    x = torch.randn(tokens, k, generator=g, device="cuda", dtype=torch.float32)
    x *= 1.0 + 4.0 * (torch.rand(k, generator=g, device="cuda") < 0.005)
    scale = x.abs().amax(1) / 127.0
    q = (x / scale[:, None]).round_().clamp_(-127, 127).to(torch.int8)
    return _packed(q), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, tokens, k = case["op"], case["tokens"], case["k"]
    dtype = DTYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype, "act": case.get("act")}
    if op == "quantize":
        x = torch.randn(tokens, k, generator=g, device="cuda", dtype=torch.float32)
        x *= 1.0 + 4.0 * (torch.rand(k, generator=g, device="cuda") < 0.005)
        s["x"] = x.to(dtype)
        return s
    rows = case["rows"]
    s["x"], s["x_scale"] = _activations(tokens, k, g)
    s["w"], s["w_scale"] = _weights(rows, k, g)
    if op == "matmul":
        s["bias"] = torch.randn(rows, generator=g, device="cuda") if case["bias"] else None
        return s
    s["w_up"], s["up_scale"] = _weights(rows, k, g)
    if op == "backward":
        s["d_out"] = torch.randn(tokens, rows, generator=g, device="cuda").to(dtype)
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


def _act_and_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if act == "relu":
        return _act(g, act), (g > 0).to(g.dtype)
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _values(packed):
    return packed.view(torch.int8).float()


def _quantize(x):
    x = x.float()
    top = x.abs().amax(1)
    small = top < TINY
    # 127 / top and top / 127 as f32 quotients (through 64 bits, rounded once)
    wide = top.double()
    inverse = torch.where(small, torch.zeros_like(wide), torch.div(torch.full_like(wide, 127.0), wide)).float()
    scale = torch.where(small, torch.zeros_like(wide), torch.div(wide, torch.full_like(wide, 127.0))).float()
    return (x * inverse[:, None]).round().to(torch.int8), scale


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        return _quantize(s["x"])
    x, xs = _values(s["x"]), s["x_scale"][:, None]
    w = _values(s["w"])
    acc = x @ w.t()
    g = acc * s["w_scale"] * xs
    if op == "matmul":
        return (g if s["bias"] is None else g + s["bias"]).to(s["dtype"])
    v = _values(s["w_up"])
    acc_up = x @ v.t()
    u = acc_up * s["up_scale"] * xs
    if op == "gated":
        return (_act(g, s["act"]) * u).to(s["dtype"])
    a, slope = _act_and_slope(g, s["act"])
    d = s["d_out"].float()
    dg, du = d * u * slope, d * a
    d_x = (dg * s["w_scale"]) @ w + (du * s["up_scale"]) @ v
    return d_x.to(s["dtype"]), (dg * acc * xs).sum(0), (du * acc_up * xs).sum(0)


def _run_own(s):
    import int8_dequant_dot_amd as loom

    op = s["op"]
    if op == "quantize":
        q, scale = loom.quantize_rows(s["x"])
        return q.view(torch.int8), scale
    if op == "matmul":
        return loom.i8_matmul(s["w"], s["w_scale"], s["x"], s["x_scale"], bias=s["bias"], dtype=s["dtype"])
    if op == "gated":
        return loom.i8_gated_projection(s["w"], s["w_scale"], s["w_up"], s["up_scale"], s["x"], s["x_scale"],
                                        act=s["act"], dtype=s["dtype"])
    return loom.i8_gated_projection_backward(s["w"], s["w_scale"], s["w_up"], s["up_scale"], s["x"], s["x_scale"],
                                             s["d_out"], act=s["act"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the work and the 64-bit values

def work(case):
    t, k, b = case["tokens"], case["k"], {"float32": 4}.get(case["dtype"], 2)
    if case["op"] == "quantize":
        return {"bytes": t * k * (b + 1) + 4 * t, "flops": 3 * t * k}
    n = case["rows"]
    one = 2 * t * n * k
    if case["op"] == "matmul":
        return {"bytes": n * k + t * k + 4 * (n + t) + t * n * b + (4 * n if case["bias"] else 0), "flops": one}
    if case["op"] == "gated":
        return {"bytes": 2 * n * k + t * k + 4 * (2 * n + t) + t * n * b, "flops": 2 * one}
    # both products again (the projections are not kept), and the gradients through both
    return {"bytes": 2 * n * k + t * k + 4 * (4 * n + t) + t * n * b + t * k * b, "flops": 4 * one}


def exact(case, seed):
    """The definitions in float64: sums of products of the integers, the scales, the activation and its derivative."""
    s = prepare(case, seed)
    act = s["act"]
    if s["op"] == "quantize":
        # the scale is the f32 nearest to max/127, the reciprocal the f32 nearest to 127/max
        x = s["x"].to(torch.float64)
        peak = torch.maximum(x.amax(dim=1), -x.amin(dim=1))
        n127 = torch.full_like(peak, 127.0)
        live = peak >= TINY
        r = torch.where(live, (n127 / peak).float().double(), 0.0)
        q = torch.round((x * r.unsqueeze(1)).float())
        return q.to(torch.int8), torch.where(live, peak / n127, 0.0)
    x = s["x"].view(torch.int8).to(torch.float64) * s["x_scale"].double().unsqueeze(1)
    wg = s["w"].view(torch.int8).to(torch.float64)
    pre_g = torch.mm(x, wg.t().contiguous())
    g = pre_g * s["w_scale"].double().unsqueeze(0)
    if s["op"] == "matmul":
        return g if s["bias"] is None else g + s["bias"].double()
    wu = s["w_up"].view(torch.int8).to(torch.float64)
    pre_u = torch.mm(x, wu.t().contiguous())
    u = pre_u * s["up_scale"].double().unsqueeze(0)
    if act == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * (1 - sig)
    elif act == "relu":
        a, da = g.clamp(min=0), (g > 0).double()
    elif act == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        a, da = g * cdf, cdf + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    else:
        # tanh z = 2 sigmoid(2 z) - 1, so the factor (1 + tanh z) / 2 is sigmoid(2 z)
        z2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        sig = torch.sigmoid(z2)
        a, da = g * sig, sig + g * sig * (1 - sig) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())
    if s["op"] == "gated":
        return a * u
    d = s["d_out"].double()
    dg, du = d * da * u, d * a
    d_gate, d_up = (dg * pre_g).sum(0), (du * pre_u).sum(0)
    wg *= s["w_scale"].double().unsqueeze(1)
    wu *= s["up_scale"].double().unsqueeze(1)
    return torch.mm(dg, wg).add_(torch.mm(du, wu)), d_gate, d_up
