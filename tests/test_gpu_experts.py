"""The router, its gradient, route grouping and the 4-bit products on the GPU against plain 64-bit implementations.

Tolerances (u = 2^-24, half a step of f32; HALF is half a step of the output type; d is how far a logit lies below the
largest, which is what the rounding of the exponent l - max costs, in units of u):
 - expf is within 2 u, a quotient or sum within u.  A softmax's sum carries the terms' errors (2 u, and the mean of d over
   the softmax, at most ln 1024 < 7) and at most 16 additions in a lane and 6 across: (d + 2) + 31 + 2 < d + 40.
 - a sigmoid is one exponential, a sum and a quotient: 4 u; renormalised weights are quotients of such terms and a sum of
   at most 64 of them (at most 6 additions deep): 2 d + 32.
 - gradients are products of these with differences whose parts are bounded by the sums of magnitudes: 2 d + 64 (4 d + 64
   renormalised) times those sums.
 - the 4-bit product adds groups, and parts of 128 of longer groups, whose sums are exact in int32: a part's conversion is
   within u, and each of the n additions rounds a partial sum that is at most the sum of the parts' magnitudes: (n + 8) u
   times that sum, n the parts, then one u for x_scale and one for the bias.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: U, F16: 2.0 ** -11, BF16: 2.0 ** -8}
LOW = {F32: 2.0 ** -126, F16: 2.0 ** -25, BF16: 2.0 ** -126}  # flushed or subnormal results
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


# ------------------------------------------------------------------ the router

def scores64(l, score):
    if score == "sigmoid":
        return torch.sigmoid(l)
    return torch.softmax(l, 1)


def route_ref(logits, top_k, score, bias, groups, top_groups, group_top, renormalize, scale):
    """By the definition, token by token -> (ids, weights in float64)."""
    l = logits.double()
    tokens, experts = l.shape
    s = torch.nan_to_num(scores64(l, score), nan=0.0)
    choice = l if bias is None else s + bias.double()
    choice = torch.where(l == -INF, torch.full_like(l, -INF), choice)
    ids = np.full((tokens, top_k), -1, np.int32)
    w = np.zeros((tokens, top_k))
    size = experts // groups
    for t in range(tokens):
        if bool((~(l[t] < INF)).any()) or bool(((l[t] > -INF) & choice[t].isnan()).any()):
            ids[t], w[t] = np.arange(top_k), NAN
            continue
        c = choice[t].tolist()
        if groups > 1:
            rank = []
            for g in range(groups):
                v = c if bias is not None or group_top == 1 else [x if y > -INF else -INF for x, y in zip(s[t].tolist(), c)]
                v = sorted((x for x in v[g * size:(g + 1) * size] if x > -INF), reverse=True)[:group_top]
                rank.append(sum(v) if v else -INF)
            kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            c = [x if e // size in kept else -INF for e, x in enumerate(c)]
        order = [e for e in sorted(range(experts), key=lambda e: (-c[e], e)) if c[e] > -INF][:top_k]
        ids[t, :len(order)] = order
        if not order:
            continue
        chosen = l[t, order]
        if renormalize:  # of logarithms, so that vanishing scores keep their ratio
            log = chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen)
            r = torch.softmax(log, 0)
        else:
            r = s[t, order]
        w[t, :len(order)] = (scale * r).numpy()
    return ids, w


def route_tolerance(logits, ids, w, score, renormalize):
    l = logits.double()
    top = l.max(1, keepdim=True).values
    at = torch.gather(l, 1, torch.from_numpy(ids).long().clamp(min=0))
    d = (top - at).abs().nan_to_num(0, 0, 0)
    if renormalize:
        d = 2 * (d + (at.abs().nan_to_num(0, 0, 0) if score == "sigmoid" else 0)) - 8
    elif score == "sigmoid":
        d = 0 * d
    return (d + 40).numpy() * U * np.abs(w) + LOW[F32]


def check_route(loom, device, logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_top=2,
                renormalize=True, scale=1.0):
    ids, w = loom.route_experts(logits, top_k, score=score, bias=None if bias is None else bias.to(device), groups=groups,
                                top_groups=top_groups, group_top=group_top, renormalize=renormalize, scale=scale)
    assert ids.dtype == torch.int32 and w.dtype == F32 and tuple(ids.shape) == tuple(w.shape) == (logits.shape[0], top_k)
    host = logits.cpu()
    rids, rw = route_ref(host, top_k, score, bias, groups, top_groups, group_top, renormalize, scale)
    assert np.array_equal(ids.cpu().numpy(), rids)
    got = w.cpu().numpy().astype(np.float64)
    if rw.size:
        assert np.array_equal(np.isnan(got), np.isnan(rw))
        tol = route_tolerance(host, rids, np.nan_to_num(rw), score, renormalize)
        assert np.all(np.abs(np.nan_to_num(got) - np.nan_to_num(rw)) <= tol)


ROUTES = [(1, 8, 1, 1, 1, 1), (3, 60, 4, 1, 1, 1), (5, 64, 6, 8, 3, 2), (2, 256, 8, 8, 4, 2), (7, 256, 16, 4, 2, 1),
          (1, 1024, 64, 16, 9, 2), (4, 1000, 10, 50, 7, 1), (9, 17, 17, 1, 1, 2), (6, 128, 32, 64, 33, 2), (2, 1, 1, 1, 1, 2),
          (1030, 64, 8, 8, 4, 2), (1100, 256, 8, 8, 4, 2), (1025, 100, 5, 10, 3, 1), (1041, 200, 3, 1, 1, 2),
          (1024, 15, 15, 3, 3, 2), (1200, 40, 2, 40, 20, 2), (0, 16, 2, 1, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups,group_top", ROUTES)
def test_route(loom, device, tokens, experts, top_k, groups, top_groups, group_top, biased, score):
    g = torch.Generator().manual_seed(tokens * 7 + experts)
    logits = 2 * torch.randn(tokens, experts, generator=g)
    bias = 0.1 * torch.randn(experts, generator=g) if biased else None
    for dtype, renormalize in ((F32, True), (BF16, False), (F16, True)):
        check_route(loom, device, logits.to(dtype).to(device), top_k, score, bias, groups, top_groups, group_top, renormalize,
                    2.5)


@pytest.mark.parametrize("tokens", [33, 1500])
def test_route_ties(loom, device, tokens):
    """Few distinct logits: nearly every place is a tie, also between groups, and with equal biases."""
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-2, 3, (tokens, 96), generator=g).float()
    for score in ("softmax", "sigmoid"):
        check_route(loom, device, logits.to(device), 8, score)
        check_route(loom, device, logits.to(BF16).to(device), 8, score, None, 8, 3, 1, False)
        check_route(loom, device, logits.to(device), 7, score, None, 12, 5, 2)
        check_route(loom, device, logits.to(device), 8, score, torch.full((96,), 0.25), 8, 3, 2)


@pytest.mark.parametrize("tokens", [5, 1300])
def test_route_near_ties(loom, device, tokens):
    """Choices that differ by less than a step of f32: only their 64-bit values order them."""
    g = torch.Generator().manual_seed(8)
    experts = 64
    logits = (1 + torch.randint(0, 3, (tokens, experts), generator=g) * 2.0 ** -23).float()
    bias = torch.zeros(experts)
    bias[::3] = 2.0 ** -26
    for score in ("softmax", "sigmoid"):
        check_route(loom, device, logits.to(device), 8, score, bias)
        check_route(loom, device, logits.to(device), 8, score, bias, 8, 4, 2)
        check_route(loom, device, logits.to(device), 8, score, None, 8, 4, 2)


@pytest.mark.parametrize("tokens", [8, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_special(loom, device, score, tokens):
    """Masked experts, masked groups, rows without any, the lowest finite value, NaN and infinities, far logits."""
    g = torch.Generator().manual_seed(11)
    experts = 48
    l = 3 * torch.randn(tokens, experts, generator=g)
    l[0] = -INF
    l[1, 3:] = -INF
    l[2, :40] = -INF
    l[3] = torch.finfo(F32).min
    l[3, 5] = -200.0
    l[4, 17] = NAN
    l[5, 47] = INF
    l[6] = -120 - torch.arange(experts) * 0.5
    l[7] = 90 + torch.arange(experts) * 0.25
    bias = 0.1 * torch.randn(experts, generator=g)
    for groups, kept in ((1, 1), (6, 2)):
        for top in (1, 2):
            for renormalize in (True, False):
                check_route(loom, device, l.to(device), 6, score, None, groups, kept, top, renormalize)
                check_route(loom, device, l.to(device), 6, score, bias, groups, kept, top, renormalize)
    shut = bias.clone()
    shut[4], shut[9] = -INF, INF
    check_route(loom, device, l.to(device), 6, score, shut, 6, 2, 2)
    shut[9] = NAN
    check_route(loom, device, l.to(device), 6, score, shut)


def test_route_strided(loom, device):
    """Strided logits at odd offsets, given outputs that are longer than needed."""
    for tokens in (6, 1200):
        for dtype in (F32, BF16, F16):
            g = torch.Generator().manual_seed(2)
            base = torch.randn(tokens, 77, generator=g).to(dtype).to(device)
            logits = base[:, 3:67]
            check_route(loom, device, logits, 5, "sigmoid", 0.1 * torch.randn(64, generator=g), 4, 2, 2)
            ids = torch.full((tokens * 5 + 3,), 99, dtype=torch.int32, device=device)
            w = torch.full((tokens * 5 + 3,), 9.0, device=device)
            a, b = loom.route_experts(logits, 5, ids=ids, weights=w)
            assert a is ids and b is w
            i2, w2 = loom.route_experts(logits, 5)
            assert torch.equal(ids[:-3], i2.flatten()) and torch.equal(w[:-3], w2.flatten())
            assert bool((ids[-3:] == 99).all()) and bool((w[-3:] == 9.0).all())


# ------------------------------------------------------------------ its gradient

def backward_ref(logits, ids, d, score, renormalize, scale):
    """-> (gradient, the sum of magnitudes it is made of, the reach d of the exponents), float64."""
    l = logits.double()
    tokens, experts = l.shape
    out, size = torch.zeros_like(l), torch.zeros_like(l)
    s = scores64(l, score)
    for t in range(tokens):
        live = [i for i in range(ids.shape[1]) if 0 <= int(ids[t, i]) < experts]
        if not live:
            continue
        e, a = ids[t, live].long(), scale * d[t, live].double()
        if renormalize:
            log = l[t, e] if score == "softmax" else torch.nn.functional.logsigmoid(l[t, e])
            w = torch.softmax(log, 0)
            slope = torch.ones_like(w) if score == "softmax" else torch.sigmoid(-l[t, e])
            out[t].index_add_(0, e, w * (a - (w * a).sum()) * slope)
            size[t].index_add_(0, e, w * (a.abs() + (w * a.abs()).sum()) * slope)
        elif score == "sigmoid":
            out[t].index_add_(0, e, a * s[t, e] * (1 - s[t, e]))
            size[t].index_add_(0, e, a.abs() * s[t, e] * (1 - s[t, e]))
        else:
            out[t] = -s[t] * (s[t, e] * a).sum()
            size[t] = s[t] * (s[t, e] * a.abs()).sum()
            out[t].index_add_(0, e, s[t, e] * a)
            size[t].index_add_(0, e, s[t, e] * a.abs())
    return out, size


def check_backward(loom, device, logits, ids, d, score, renormalize, scale=2.5, **kw):
    got = loom.route_experts_backward(logits, ids.to(device), d.to(device), score=score, renormalize=renormalize,
                                      scale=scale, **kw)
    host = logits.cpu()
    ref, size = backward_ref(host, ids, d, score, renormalize, scale)
    assert got.dtype == logits.dtype and got.shape == logits.shape
    if not ref.numel():
        return
    l = host.double()
    far = (l.max(1, keepdim=True).values - l).nan_to_num(0).clamp(max=200)
    if score == "sigmoid":
        far = far + l.abs().clamp(max=200)
    tol = (4 * far + 64) * U * size + HALF[logits.dtype] * ref.abs() + LOW[logits.dtype]
    assert bool(((got.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 8, 1), (3, 60, 4), (2, 256, 8), (1, 1024, 64), (5, 17, 17),
                                                  (1030, 64, 6), (1100, 256, 16), (1024, 5, 3), (1025, 100, 1), (0, 8, 2)])
def test_backward(loom, device, tokens, experts, top_k, score, renormalize):
    g = torch.Generator().manual_seed(tokens + experts)
    logits = 2 * torch.randn(tokens, experts, generator=g)
    ids = torch.topk(logits, top_k, dim=1).indices.to(torch.int32)
    d = torch.randn(tokens, top_k, generator=g)
    for dtype in (F32, BF16, F16):
        check_backward(loom, device, logits.to(dtype).to(device), ids, d, score, renormalize)


@pytest.mark.parametrize("tokens", [7, 1200])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_odd_ids(loom, device, score, renormalize, tokens):
    """Missing routes (whose gradient is NaN and not read), tokens without any, the same expert named twice and three
    times, masked logits, strided rows; every logit that is not written stays."""
    g = torch.Generator().manual_seed(4)
    experts, top_k = 40, 6
    logits = 2 * torch.randn(tokens, experts, generator=g)
    logits[:, 7] = -INF
    ids = torch.topk(logits, top_k, dim=1).indices.to(torch.int32)
    d = torch.randn(tokens, top_k, generator=g)
    ids[0] = -1
    ids[1, 2:] = torch.tensor([experts, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    ids[2, 3] = ids[2, 0]
    ids[3, :] = ids[3, 0]
    ids[4, 1] = ids[4, 4] = ids[4, 5]
    logits[5] = -INF
    ids[5] = -1
    d[ids < 0] = NAN
    d[ids >= experts] = NAN
    for dtype in (F32, BF16):
        base = torch.full((tokens, experts + 9), 7.0, dtype=dtype, device=device)
        big = torch.zeros(tokens, experts + 3, dtype=dtype, device=device)
        big[:, 1:1 + experts] = logits.to(dtype).to(device)
        out = base[:, 5:5 + experts]
        check_backward(loom, device, big[:, 1:1 + experts], ids, d, score, renormalize, d_logits=out)
        assert bool((base[:, :5] == 7).all()) and bool((base[:, 5 + experts:] == 7).all())


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_against_differences(loom, device, score, renormalize):
    """Central differences of the forward pass with step h: third derivatives of these weights are at most 2 in size, so
    truncation is at most h^2 / 3 and rounding 100 u / h, times the sum of the gradients' magnitudes."""
    experts, top_k, h = 12, 4, 2.0 ** -6
    g = torch.Generator().manual_seed(1)
    logits = torch.randperm(experts, generator=g).float()[None] * 0.25 - 1.5
    d = torch.randn(1, top_k, generator=g)
    dev = logits.to(device)
    ids, _ = loom.route_experts(dev, top_k, score=score, renormalize=renormalize, scale=1.5)
    grad = loom.route_experts_backward(dev, ids, d.to(device), score=score, renormalize=renormalize, scale=1.5)[0].cpu()
    both = torch.cat([logits + h * torch.eye(experts), logits - h * torch.eye(experts)]).to(device)
    i2, w = loom.route_experts(both, top_k, score=score, renormalize=renormalize, scale=1.5)
    assert torch.equal(i2, ids.expand_as(i2))
    f = (w.cpu().double() * d.double()).sum(1)
    diff = (f[:experts] - f[experts:]) / (2 * h)
    assert bool(((diff - grad.double()).abs() <= 1.5 * d.abs().sum() * (h * h / 3 + 100 * U / h)).all())


# ------------------------------------------------------------------ grouping

def group_ref(ids, experts):
    tokens, routes = ids.shape
    flat = ids.reshape(-1).numpy()
    slots, rows, offsets = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32), np.zeros(experts + 1, np.int32)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    count = np.bincount(key, minlength=experts + 1)
    offsets[1:] = np.cumsum(count[:experts])
    n = offsets[experts]
    slots[order[:n]] = np.arange(n)
    rows[:n] = order[:n] // max(routes, 1)
    return slots.reshape(tokens, routes), rows, offsets


@pytest.mark.parametrize("tokens,routes,experts", [(1, 1, 1), (1, 8, 256), (64, 8, 256), (100, 3, 1024), (0, 4, 7), (5, 0, 3),
                                                   (512, 8, 8), (513, 8, 60), (1365, 3, 100), (4097, 1, 2), (3000, 6, 1000),
                                                   (60000, 8, 256), (200001, 7, 1024), (1500000, 1, 33)])
def test_group_routes(loom, device, tokens, routes, experts):
    g = torch.Generator().manual_seed(tokens + routes)
    for spread in ("even", "one", "missing"):
        ids = torch.randint(0, experts, (tokens, routes), generator=g, dtype=torch.int32)
        if spread == "one":
            ids[:] = experts - 1
        if spread == "missing":
            odd = torch.rand(tokens, routes, generator=g)
            ids[odd < 0.2], ids[odd > 0.9] = -1, experts
            ids[(odd > 0.5) & (odd < 0.52)] = 2 ** 31 - 1
            ids[(odd > 0.6) & (odd < 0.62)] = -2 ** 31
        got = loom.group_routes(ids.to(device), experts)
        for a, b in zip(got, group_ref(ids, experts)):
            assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b)


def test_group_routes_buffers(loom, device):
    """Given buffers that are larger than needed keep what lies behind; the workspace's old contents do not matter."""
    ids = torch.randint(-1, 50, (3000, 5), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    want = group_ref(ids, 50)
    n = 15000
    need = loom.group_routes_workspace(3000, 5, 50)
    assert need > 0
    for fill in (0, 255):
        slots, rows, offsets = (torch.full((m + 2,), 77, dtype=torch.int32, device=device) for m in (n, n, 51))
        space = torch.full((need,), fill, dtype=torch.uint8, device=device)
        loom.group_routes(ids.to(device), 50, slots, rows, offsets, space)
        for a, b in zip((slots, rows, offsets), want):
            assert np.array_equal(a.cpu().numpy()[:-2], b.reshape(-1)) and bool((a[-2:] == 77).all())
    with pytest.raises(ValueError):
        loom.group_routes(ids.to(device), 50, workspace=torch.empty(need - 1, dtype=torch.uint8, device=device))


# ------------------------------------------------------------------ the 4-bit products

def operands(experts, rows, k, x_rows, group, scales, seed, names=("w",)):
    g = torch.Generator().manual_seed(seed)
    s = {}
    for n in names:
        s[n] = torch.randint(-8, 8, (experts, rows, k), generator=g, dtype=torch.int8)
        s[n + "s"] = ((0.5 + torch.rand(experts, rows, -(-k // group), generator=g)) / (5 * 74 * max(1.0, math.sqrt(k)))).to(scales)
    s["x"] = torch.randint(-128, 128, (x_rows, k), generator=g, dtype=torch.int8)
    s["xs"] = 0.02 + 0.08 * torch.rand(x_rows, generator=g)
    s["bias"] = torch.randn(experts, rows, generator=g)
    return s


def product64(x, w, ws, group):
    """-> (sum over groups of scale * sum, the same sum of magnitudes of groups and parts of 128 of longer ones)."""
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    size = y.clone()
    step = min(group, 128)
    for at in range(0, x.shape[1], step):
        part = slice(at, at + step)
        term = (x[:, part].double() @ w[:, part].double().t()) * ws[:, at // group].double()
        y += term
        size += term.abs()
    return y, size


def parts(k, group):
    return -(-k // min(group, 128))


def bounded(y, size, groups, xs, bias, dtype):
    """-> (the value, its tolerance); groups: how many parts are added."""
    v, s = (y, size) if xs is None else (y * xs.double()[:, None], size * xs.double()[:, None].abs())
    tol = (groups + 10) * U * s
    if bias is not None:
        v = v + bias.double()
        tol = tol + U * v.abs() + U * s
    return v, tol * (1 + 2 * HALF[dtype]) + HALF[dtype] * v.abs() + LOW[dtype]


def check(got, v, tol):
    assert bool(((got.cpu().double() - v).abs() <= tol).all())


SHAPES = [(1, 32, 1, 32), (1, 8192, 1, 128), (17, 64, 1, 32), (64, 256, 3, 64), (33, 1056, 16, 32), (130, 96, 17, 64),
          (16, 512, 2, 128), (15, 2016, 4, 256), (48, 1024, 5, 1024), (100, 3328, 8, 32), (257, 544, 65, 64),
          (300, 1024, 130, 32), (256, 2048, 64, 128), (255, 160, 31, 32), (512, 128, 256, 128), (513, 192, 257, 32),
          (129, 4096, 129, 64), (1030, 320, 33, 128), (77, 11008, 9, 32), (2100, 288, 7, 64), (640, 1024, 512, 256),
          (31, 64, 1000, 32), (384, 32, 300, 131072), (8, 16416, 12, 128), (70, 131040, 3, 131072), (70, 65536, 20, 32),
          (1500, 512, 700, 128), (96, 0, 5, 32), (40, 4192, 21, 512), (1000, 768, 4, 32), (1000, 768, 40, 128)]


@pytest.mark.parametrize("rows,k,tokens,group", SHAPES)
def test_i4_matmul(loom, device, rows, k, tokens, group):
    for dtype, scales in ((F32, F32), (BF16, F16), (F16, BF16)):
        s = operands(1, rows, k, tokens, group, scales, rows + k + tokens)
        d = {n: t.to(device) for n, t in s.items()}
        y, size = product64(s["x"], s["w"][0], s["ws"][0], group)
        n = parts(k, group)
        w, x = loom.pack_int4(d["w"][0]), loom.pack_int8(d["x"])
        got = loom.i4_matmul(w, d["ws"][0], x, d["xs"], bias=d["bias"][0], group=group, dtype=dtype)
        assert got.dtype == dtype and tuple(got.shape) == (tokens, rows)
        check(got, *bounded(y, size, n, s["xs"], s["bias"][0], dtype))
        check(loom.i4_matmul(w, d["ws"][0], x, group=group, dtype=F32), *bounded(y, size, n, None, None, F32))


@pytest.mark.parametrize("tokens", [1, 3, 8, 16, 17, 40, 64, 90, 128, 300])
def test_i4_matmul_one_hot(loom, device, tokens):
    """Each nibble of a row, one at a time, against distinct values: order, sign, every k position and its scale."""
    k = 1120
    g = torch.Generator().manual_seed(tokens)
    x = torch.randint(-128, 128, (tokens, k), generator=g, dtype=torch.int8)
    for value in (-8, -1, 7):
        w = torch.eye(k, dtype=torch.int8) * value
        for group in (32, 64, 128, 256):
            scale = (1 + torch.arange(k // group + (k % group > 0))).float().expand(k, -1).contiguous()
            got = loom.i4_matmul(loom.pack_int4(w.to(device)), scale.to(device), loom.pack_int8(x.to(device)), group=group, dtype=F32)
            assert torch.equal(got.cpu(), value * x.float() * (1 + torch.arange(k) // group))


def test_i4_matmul_limits(loom, device):
    """The accumulator's limits: -128 against -8 and 127 against -8 over the longest row as one group."""
    k = 131040
    for tokens in (1, 20, 70, 200):
        for a, b in ((-8, -128), (-8, 127), (7, -128)):
            w = torch.full((65, k), a, dtype=torch.int8, device=device)
            x = torch.full((tokens, k), b, dtype=torch.int8, device=device)
            got = loom.i4_matmul(loom.pack_int4(w), torch.ones(65, 1, device=device), loom.pack_int8(x), group=131072, dtype=F32)
            assert bool(((got.double() / (a * b * k) - 1).abs() <= 4 * U).all())


def test_i4_matmul_views_and_scales(loom, device):
    """Operands in the middle of larger ones, strided outputs (whose gaps stay), special scales, a 1-d activation."""
    for rows, k, tokens, group in ((50, 1056, 3, 32), (50, 1024, 3, 128), (140, 1184, 40, 64), (70, 256, 100, 128),
                                   (300, 2048, 300, 128)):
        s = operands(1, rows, k, tokens, group, F32, 5)
        d = {n: t.to(device) for n, t in s.items()}
        y, size = product64(s["x"], s["w"][0], s["ws"][0], group)
        n = parts(k, group)
        w, x = loom.pack_int4(d["w"][0]), loom.pack_int8(d["x"])
        wb = torch.full((rows * k // 8 + 8,), -1, dtype=torch.int32, device=device)
        xb = torch.full((tokens * k // 4 + 8,), -1, dtype=torch.int32, device=device)
        w2, x2 = wb[4:4 + w.numel()].view_as(w), xb[4:4 + x.numel()].view_as(x)
        w2.copy_(w), x2.copy_(x)
        for off in (0, 1, 2, 3):
            for dtype in (F32, BF16):
                big = torch.full((tokens, rows + 5 + off), 7.0, dtype=dtype, device=device)
                out = big[:, 2 + off:2 + off + rows]
                assert loom.i4_matmul(w2, d["ws"][0], x2, d["xs"], group=group, out=out) is out
                check(out, *bounded(y, size, n, s["xs"], None, dtype))
                assert bool((big[:, :2 + off] == 7).all()) and bool((big[:, 2 + off + rows:] == 7).all())
        xs = s["xs"].clone()
        xs[0], xs[1], xs[2] = NAN, INF, 0.0
        got = loom.i4_matmul(w, d["ws"][0], x, xs.to(device), group=group, dtype=F32).cpu()
        assert bool(got[0].isnan().all()) and bool((got[2] == 0).all()) and not bool(got[1].isfinite().any())
        check(got[3:], *(t[3:] for t in bounded(y, size, n, xs.nan_to_num(0, 0, 0), None, F32)))
        # a NaN scale of a group reaches its channel and no other
        ws = s["ws"][0].clone()
        ws[rows // 2, -1] = NAN
        got = loom.i4_matmul(w, ws.to(device), x, group=group, dtype=F32).cpu()
        assert bool(got[:, rows // 2].isnan().all()) and int(got.isnan().sum()) == tokens
    one = loom.i4_matmul(w, d["ws"][0], x[0], group=group, dtype=F32)
    check(one, *(t[:1] for t in bounded(y, size, n, None, None, F32)))


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "relu":
        return g.clamp(min=0)
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


# rows of each expert, channels, row length, group
EXPERTS = [([1], 16, 64, 32), ([0, 3, 0, 1], 40, 512, 128), ([2] * 9, 100, 1056, 32), ([0] * 70 + [5, 0, 17, 1], 33, 288, 64),
           ([64, 0, 1, 33], 257, 544, 64), ([200, 130, 0, 7], 130, 1024, 128), ([1, 0, 2, 0] * 60, 24, 2048, 128),
           ([0, 0, 0], 20, 96, 32), ([1000, 3], 70, 320, 256), ([12, 40, 90, 300] * 3, 300, 256, 128), ([5, 9], 24, 0, 32),
           ([16] * 1024, 8, 64, 32), ([31, 32, 33, 0, 128, 129], 160, 4224, 32)]


@pytest.mark.parametrize("counts,rows,k,group", EXPERTS)
def test_experts(loom, device, counts, rows, k, group):
    """Plain and gated, with and without an index, rows behind the last route left as they were."""
    experts, pairs, used = len(counts), sum(counts) + 5, sum(counts)
    offsets = offsets_of(counts)
    g = torch.Generator().manual_seed(rows + k)
    for dtype, scales, act in ((F32, F16, "silu"), (BF16, F32, "gelu"), (F16, BF16, "relu"), (F32, F32, "gelu_tanh")):
        s = operands(experts, rows, k, pairs, group, scales, rows * 3 + k, ("w", "u"))
        n = parts(k, group)
        d = {m: t.to(device) for m, t in s.items()}
        w, u, x = loom.pack_int4(d["w"]), loom.pack_int4(d["u"]), loom.pack_int8(d["x"])
        index = torch.randint(0, pairs, (pairs,), generator=g, dtype=torch.int32) if act in ("silu", "relu") else None
        xr = s["x"] if index is None else s["x"][index.long()]
        xs = s["xs"] if index is None else s["xs"][index.long()]
        out = torch.full((pairs, rows + 3), 7.0, dtype=dtype, device=device)
        gated = out.clone()
        ix = None if index is None else index.to(device)
        loom.i4_expert_matmul(w, d["ws"], x, d["xs"], offsets.to(device), index=ix, bias=d["bias"], group=group, out=out[:, :rows])
        loom.i4_expert_gated_projection(w, d["ws"], u, d["us"], x, d["xs"], offsets.to(device), index=ix, act=act, group=group,
                                        out=gated[:, 1:1 + rows])
        for b, at in ((out, slice(0, rows)), (gated, slice(1, 1 + rows))):
            rest = b.clone()
            rest[:used, at] = 7.0
            assert bool((rest == 7).all())
        for e in range(experts):
            a, b = int(offsets[e]), int(offsets[e + 1])
            if a == b:
                continue
            y, size = product64(xr[a:b], s["w"][e], s["ws"][e], group)
            check(out[a:b, :rows], *bounded(y, size, n, xs[a:b], s["bias"][e], dtype))
            yu, size_u = product64(xr[a:b], s["u"][e], s["us"][e], group)
            gv, gt = bounded(y, size, n, xs[a:b], None, F32)
            uv, ut = bounded(yu, size_u, n, xs[a:b], None, F32)
            v = act64(gv, act) * uv
            # |act'| <= 1.13; act itself within (16 |g| + 5 |act|) u
            tol = (1.13 * gt + (16 * gv.abs() + 5 * act64(gv, act).abs()) * U) * (uv.abs() + ut) + act64(gv, act).abs() * ut
            check(gated[a:b, 1:1 + rows], v, tol * (1 + HALF[dtype]) + (HALF[dtype] + U) * v.abs() + LOW[dtype])


def test_experts_bad_offsets_and_index(loom, device):
    """Offsets out of order or range make rows fewer and never others; an index outside x makes its row NaN."""
    experts, rows, k, pairs = 4, 40, 256, 50
    s = operands(experts, rows, k, pairs, 128, F32, 9)
    d = {m: t.to(device) for m, t in s.items()}
    w, x = loom.pack_int4(d["w"]), loom.pack_int8(d["x"])
    for offsets, live in (([-5, 10, 20, 20, 1000], [(0, 0, 10), (1, 10, 20), (3, 20, 50)]),
                          ([30, 20, 10, 15, 12], [(2, 10, 15)]), ([60, 70, 80, 90, 100], []),
                          ([-2 ** 31, -7, 0, 50, 2 ** 31 - 1], [(2, 0, 50)])):
        out = torch.full((pairs, rows), 7.0, device=device)
        loom.i4_expert_matmul(w, d["ws"], x, d["xs"], torch.tensor(offsets, dtype=torch.int32, device=device), group=128, out=out)
        left = torch.ones(pairs, dtype=torch.bool)
        for e, a, b in live:
            y, size = product64(s["x"][a:b], s["w"][e], s["ws"][e], 128)
            check(out[a:b], *bounded(y, size, 2, s["xs"][a:b], None, F32))
            left[a:b] = False
        assert bool((out.cpu()[left] == 7).all())
    index = torch.arange(pairs, dtype=torch.int32)
    index[3], index[20], index[41], index[49] = -1, pairs, 2 ** 31 - 1, -2 ** 31
    bad = torch.zeros(pairs, dtype=torch.bool)
    bad[[3, 20, 41, 49]] = True
    out = loom.i4_expert_matmul(w, d["ws"], x, d["xs"], offsets_of([20, 2, 0, 28]).to(device), index=index.to(device), group=128,
                                dtype=F32)
    assert torch.equal(out.cpu().isnan().all(1), bad) and torch.equal(out.cpu().isnan().any(1), bad)
    out = loom.i4_expert_gated_projection(w, d["ws"], w, d["ws"], x, None, offsets_of([20, 2, 0, 28]).to(device),
                                          index=index.to(device), group=128, act="relu", dtype=F32)
    assert torch.equal(out.cpu().isnan().all(1), bad) and torch.equal(out.cpu().isnan().any(1), bad)


def test_offsets_that_overlap(loom, device):
    """Every expert claims every row, 1024 times: rows with several claims have no defined value, the others stay."""
    experts, rows, k, pairs = 1024, 16, 64, 300
    s = operands(experts, rows, k, pairs, 64, F32, 2)
    d = {m: t.to(device) for m, t in s.items()}
    offsets = torch.tensor([0, 2 ** 31 - 1] * 512 + [0], dtype=torch.int32, device=device)
    for n in (1, 20, pairs):
        out = torch.full((pairs + 8, rows), 7.0, device=device)
        loom.i4_expert_matmul(loom.pack_int4(d["w"]), d["ws"], loom.pack_int8(d["x"][:n]), d["xs"], offsets, group=64, out=out[:n])
        assert bool((out[n:] == 7).all())


@pytest.mark.parametrize("pairs", [3, 700])
def test_weights_and_rows_past_32_bits(loom, device, pairs):
    """Weights of 5.4 GB and activations of 4.6 GB, of which the far ends are used."""
    experts, rows, k = 40, 8192, 32768
    words = torch.zeros(experts, rows, k // 8, dtype=torch.int32, device=device)
    scale = torch.ones(experts, rows, k // 256, dtype=F16, device=device)
    x_rows = 141000
    x = torch.zeros(x_rows, k // 4, dtype=torch.int32, device=device)
    g = torch.Generator().manual_seed(pairs)
    wq = torch.randint(-8, 8, (32, k), generator=g, dtype=torch.int8)
    xq = torch.randint(-128, 128, (4, k), generator=g, dtype=torch.int8)
    words[-1, -32:] = loom.pack_int4(wq.to(device))
    x[-4:] = loom.pack_int8(xq.to(device))
    index = torch.randint(x_rows - 4, x_rows, (pairs,), generator=g, dtype=torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=device)
    offsets[-1] = pairs
    out = loom.i4_expert_matmul(words, scale, x, None, offsets, index=index.to(device), group=256, dtype=F32).cpu()
    want = xq.double() @ wq.double().t()
    # whole numbers whose sums stay below 2^24
    assert torch.equal(out[:, -32:].double(), want[(index - (x_rows - 4)).long()]) and bool((out[:, :-32] == 0).all())


def test_output_past_2_31_elements(loom, device):
    rows, k, tokens = 32768, 32, 66000
    g = torch.Generator().manual_seed(1)
    wq = torch.randint(-8, 8, (rows, k), generator=g, dtype=torch.int8)
    xq = torch.randint(-128, 128, (tokens, k), generator=g, dtype=torch.int8)
    out = loom.i4_matmul(loom.pack_int4(wq.to(device)), torch.ones(rows, 1, device=device), loom.pack_int8(xq.to(device)), group=32,
                         dtype=F16)
    for at in (0, 40000, 65535, 65536, tokens - 1):
        assert torch.equal(out[at].cpu().double(), (wq.double() @ xq[at].double()).half().double())


def test_nothing_routed(loom, device):
    """No tokens, and tokens without a single route."""
    s = operands(4, 40, 64, 3, 32, F32, 1)
    w, ws, x = loom.pack_int4(s["w"].to(device)), s["ws"].to(device), loom.pack_int8(s["x"].to(device))
    none = torch.zeros(5, dtype=torch.int32, device=device)
    assert loom.i4_expert_matmul(w, ws, x[:0], None, none, group=32).shape == (0, 40)
    assert loom.i4_expert_gated_projection(w, ws, w, ws, x[:0], None, none, group=32).shape == (0, 40)
    assert loom.i4_matmul(w[0], ws[0], x[:0], group=32).shape == (0, 40)
    out = torch.full((3, 40), 7.0, device=device)
    loom.i4_expert_gated_projection(w, ws, w, ws, x, None, none, group=32, out=out)
    assert bool((out == 7).all())
    ids = torch.full((3, 2), -1, dtype=torch.int32, device=device)
    slots, rows, offsets = loom.group_routes(ids, 4)
    assert bool((slots == -1).all()) and bool((rows == -1).all()) and bool((offsets == 0).all())


def test_same_bits_every_time(loom, device):
    """No result depends on which wave comes first."""
    s = operands(6, 96, 2080, 400, 32, F16, 3, ("w", "u"))
    d = {m: t.to(device) for m, t in s.items()}
    w, u, x = loom.pack_int4(d["w"]), loom.pack_int4(d["u"]), loom.pack_int8(d["x"])
    logits = torch.randn(3000, 96, device=device)
    for n in (1, 6, 30, 400):
        off = offsets_of([n // 3, 0, n // 2, 0, 0, n - n // 3 - n // 2]).to(device)
        runs = [(loom.i4_matmul(w[0], d["ws"][0], x[:n], d["xs"], group=32, dtype=F32),
                 loom.i4_expert_gated_projection(w, d["ws"], u, d["us"], x[:n], d["xs"], off, group=32, dtype=F32))
                for _ in range(4)]
        assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
    runs = [(*loom.route_experts(logits, 5, "sigmoid", logits[0] * 0.1, 8, 4), *loom.group_routes(loom.route_experts(logits, 5)[0], 96))
            for _ in range(4)]
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


# ------------------------------------------------------------------ together

class Layer:
    def __init__(self, loom, device, experts, hidden, inner, group=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.loom, self.experts, self.group = loom, experts, group
        for name, r, k in (("gate", inner, hidden), ("up", inner, hidden), ("down", hidden, inner)):
            q = torch.randint(-8, 8, (experts, r, k), generator=g, dtype=torch.int8)
            scale = (0.5 + torch.rand(experts, r, -(-k // group), generator=g)) / (5 * math.sqrt(k))
            setattr(self, name + "_q", q), setattr(self, name + "_s", scale)
            setattr(self, name, loom.pack_int4(q.to(device))), setattr(self, name + "_scale", scale.to(device))

    def __call__(self, h, logits, bias):
        loom = self.loom
        ids, weights = loom.route_experts(logits, 4, score="sigmoid", bias=bias, groups=4, top_groups=2, scale=1.5)
        slots, rows, offsets = loom.group_routes(ids, self.experts)
        q, s = loom.quantize_rows(h)
        y = loom.i4_expert_gated_projection(self.gate, self.gate_scale, self.up, self.up_scale, q, s, offsets, index=rows,
                                            group=self.group, out=torch.zeros(rows.numel(), self.gate.shape[1], device=h.device))
        q2, s2 = loom.quantize_rows(y)
        down = loom.i4_expert_matmul(self.down, self.down_scale, q2, s2, offsets, group=self.group,
                                     out=torch.zeros(rows.numel(), self.down.shape[1], device=h.device))
        return loom.routed_combine(slots, weights, down), ids, weights, y, q2, s2


@pytest.mark.parametrize("tokens", [1, 9, 150])
def test_layer_of_experts(loom, device, tokens):
    """Router, grouping, gated projection, down projection and combine as they are used, with masked experts, against a
    layer in float64 over the same int8 activations."""
    experts, hidden, inner = 16, 256, 160
    layer = Layer(loom, device, experts, hidden, inner)
    g = torch.Generator().manual_seed(tokens)
    h = torch.randn(tokens, hidden, generator=g)
    logits = torch.randn(tokens, experts, generator=g)
    logits[:, 5] = -INF
    if tokens > 4:
        logits[2] = -INF          # a token without experts
        logits[3, 2:] = -INF      # one with fewer than it asks for
    bias = 0.1 * torch.randn(experts, generator=g)
    out, ids, weights, y, q2, s2 = layer(h.to(device), logits.to(device), bias.to(device))
    rids, rw = route_ref(logits, 4, "sigmoid", bias, 4, 2, 2, True, 1.5)
    assert np.array_equal(ids.cpu().numpy(), rids)
    q, s = (t.cpu() for t in loom.quantize_rows(h.to(device)))
    q = q.view(torch.int8)
    slots = group_ref(torch.from_numpy(rids), experts)[0]
    q2, s2 = q2.cpu().view(torch.int8), s2.cpu()
    want, tol = torch.zeros(tokens, hidden, dtype=torch.float64), torch.zeros(tokens, hidden, dtype=torch.float64)
    for t in range(tokens):
        for i in range(4):
            e, at = int(rids[t, i]), int(slots[t, i])
            if e < 0:
                continue
            gv, gt = bounded(*product64(q[t:t + 1], layer.gate_q[e], layer.gate_s[e], 64), 4, s[t:t + 1], None, F32)
            uv, ut = bounded(*product64(q[t:t + 1], layer.up_q[e], layer.up_s[e], 64), 4, s[t:t + 1], None, F32)
            v = act64(gv, "silu") * uv
            check(y[at:at + 1], v, (1.13 * gt + 21 * gv.abs() * U) * (uv.abs() + ut) + gv.abs() * ut + 2 * U * v.abs() + LOW[F32])
            dv, dt = bounded(*product64(q2[at:at + 1], layer.down_q[e], layer.down_s[e], 64), 3, s2[at:at + 1], None, F32)
            want[t] += float(rw[t, i]) * dv[0]
            # the weight's own error (an exponent's reach of at most 20), the product's and the sum's roundings
            tol[t] += float(rw[t, i]) * (dt[0] + 90 * U * dv[0].abs())
    assert bool(((out.cpu().double() - want).abs() <= tol + LOW[F32]).all())
    if tokens > 4:
        assert bool((out[2] == 0).all())


def test_layer_in_a_graph(loom, device):
    """The whole layer captured once and replayed over new inputs, with eager work between, gives the eager bits."""
    layer = Layer(loom, device, 16, 256, 160, seed=1)
    h, logits, bias = torch.randn(70, 256, device=device), torch.randn(70, 16, device=device), 0.1 * torch.randn(16, device=device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(h, logits, bias)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(h, logits, bias)
    for step in range(4):
        h.normal_(), logits.normal_()
        want = layer(h, logits, bias)
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), step
        (torch.randn(1000, 1000, device=device) @ torch.randn(1000, 1000, device=device)).sum().item()


def test_backward_and_grouping_in_graphs(loom, device):
    """The gradient and the grouping in several parts, captured in two graphs of the same buffers, replayed in turn."""
    logits, d = torch.randn(2000, 64, device=device), torch.randn(2000, 6, device=device)
    ids, _ = loom.route_experts(logits, 6)
    graphs = []
    for score in ("softmax", "sigmoid"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = (loom.route_experts_backward(logits, ids, d, score=score, renormalize=False), *loom.group_routes(ids, 64))
        graphs.append((score, graph, out))
    for step in range(3):
        logits.normal_(), d.normal_()
        loom.route_experts(logits, 6, ids=ids)
        for score, graph, out in graphs + graphs[::-1]:
            graph.replay()
            want = (loom.route_experts_backward(logits, ids, d, score=score, renormalize=False), *loom.group_routes(ids, 64))
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams(loom, device):
    """Calls of the same sizes on two streams at once do not meet."""
    layers = [Layer(loom, device, 16, 256, 160, seed=s) for s in (2, 3)]
    h = [torch.randn(64, 256, device=device) for _ in layers]
    logits, bias = torch.randn(64, 16, device=device), 0.1 * torch.randn(16, device=device)
    want = [layer(x, logits, bias)[0] for layer, x in zip(layers, h)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        got = []
        for layer, x, stream in zip(layers, h, streams):
            with torch.cuda.stream(stream):
                got.append(layer(x, logits, bias)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(loom, device):
    l = torch.randn(4, 16, device=device)
    E = loom.LoomError
    ids, w = loom.route_experts(l, 2)
    for kw in (dict(top_k=0), dict(top_k=65), dict(top_k=17), dict(top_k=2, groups=3), dict(top_k=2, groups=0), dict(top_k=2, group_top=3),
               dict(top_k=2, groups=4, top_groups=5), dict(top_k=5, groups=4, top_groups=1)):
        with pytest.raises(E):
            loom.route_experts(l, **kw)
    with pytest.raises(ValueError):
        loom.route_experts(l, 2, score="tanh")
    with pytest.raises(ValueError):
        loom.route_experts(l, 2, bias=torch.zeros(15, device=device))
    with pytest.raises(TypeError):
        loom.route_experts(l.double(), 2)
    with pytest.raises(ValueError):
        loom.route_experts(l.t(), 2)
    with pytest.raises(TypeError):
        loom.route_experts_backward(l, ids.long(), w)
    with pytest.raises(ValueError):
        loom.route_experts_backward(l, ids[:3], w)
    with pytest.raises(ValueError):
        loom.route_experts_backward(l, ids, w[:, :1])
    with pytest.raises(E):
        loom.group_routes(ids, 0)
    with pytest.raises(E):
        loom.group_routes(ids, 1025)
    q = loom.pack_int4(torch.zeros(8, 64, dtype=torch.int8, device=device))
    x = loom.pack_int8(torch.zeros(3, 64, dtype=torch.int8, device=device))
    s = torch.ones(8, 2, device=device)
    for group in (16, 48, 2 ** 18):
        with pytest.raises((E, ValueError)):
            loom.i4_matmul(q, torch.ones(8, 4, device=device), x, group=group)
    with pytest.raises(ValueError):
        loom.i4_matmul(q, s[:, :1].contiguous(), x, group=32)
    with pytest.raises(TypeError):
        loom.i4_matmul(q, s.double(), x, group=32)
    with pytest.raises(ValueError):
        loom.i4_matmul(q, s, x[:, :8].contiguous(), group=32)
    with pytest.raises(E):  # 4-byte aligned only
        loom.i4_matmul(torch.zeros(65, dtype=torch.int32, device=device)[1:].view(8, 8), s, x, group=32)
    with pytest.raises(E):  # k is no multiple of 32
        loom.i4_matmul(q[:, :6].contiguous(), s, loom.pack_int8(torch.zeros(3, 48, dtype=torch.int8, device=device)), group=32)
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=device)
    q3, s3 = torch.stack([q, q]), torch.stack([s, s])
    with pytest.raises(ValueError):
        loom.i4_expert_matmul(q3, s3, x, None, off[:2], group=32)
    with pytest.raises(TypeError):
        loom.i4_expert_matmul(q3, s3, x, None, off.long(), group=32)
    with pytest.raises(ValueError):
        loom.i4_expert_matmul(q, s, x, None, off, group=32)
    with pytest.raises(ValueError):
        loom.i4_expert_gated_projection(q3, s3, q3, s3.half(), x, None, off, group=32)
    with pytest.raises(ValueError):
        loom.i4_expert_gated_projection(q3, s3, q3, s3, x, None, off, group=32, act="tanh")
