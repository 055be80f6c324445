"""The int8 feed-forward operators on the GPU against plain float64 and integer implementations on the CPU.

Tolerances (u = 2^-24, half a step of f32; h = half a step of the output type):
 - quantised values and scales, and the product's f32 outputs, are the documented roundings exactly; 16-bit outputs are
   those f32 values rounded once.
 - act(g) is evaluated from a g that carries 3 roundings, with a few f32 operations and library functions whose results
   are at most of size 1 and carry at most 4 u together with their argument's rounding: within (16 |g| + 5 |act(g)|) u.
   Its derivative: within (16 + 4 |g|) u.
 - sums of n f32 terms: each addition rounds a partial sum that is at most the sum of magnitudes; over n independent
   roundings the error grows as sqrt(n), so (4 + sqrt(n)) u times the sum of magnitudes.
 - the coefficients of d_x are rounded to bfloat16 (half a step: 2^-8) for bfloat16 gradients and kept to at least
   16 bits (2^-16) for float16 ones and 22 bits (2^-22) for float32 ones.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: U, F16: 2.0 ** -11, BF16: 2.0 ** -8}
LOW = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -133}  # half the smallest subnormal, or less than a step
COEF = {F32: 2.0 ** -22, F16: 2.0 ** -16, BF16: 2.0 ** -8}
TINY = 2.0 ** -119


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


# ------------------------------------------------------------------ quantize_rows

def quantize_ref(x):
    v = x.float().numpy()
    top = np.abs(v).max(1, initial=0.0).astype(np.float32)
    bad = ~np.isfinite(v).all(1)
    live = ~bad & (top >= np.float32(TINY))
    safe = np.where(live, top, np.float32(1))
    inverse = (np.float32(127) / safe).astype(np.float32)
    q = np.rint((np.where(live[:, None], v, 0) * inverse[:, None]).astype(np.float32)).astype(np.int8)
    scale = np.where(live, safe / np.float32(127), np.float32(0)).astype(np.float32)
    scale[bad] = np.nan
    return q, scale


def check_quantize(loom, device, x):
    q, scale = loom.quantize_rows(x)
    rq, rs = quantize_ref(x.cpu())
    assert q.dtype == torch.int32 and tuple(q.shape) == (x.shape[0], x.shape[1] // 4)
    if q.numel():
        assert np.array_equal(q.cpu().numpy().view(np.int8).reshape(rq.shape), rq)
    assert np.array_equal(scale.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 4), (1, 8192), (3, 12), (2, 508), (5, 1028), (65, 64), (7, 4096), (9, 11008),
                                       (3, 16388), (2, 28672), (2, 65540), (1, 131072), (300, 256), (1000, 36), (0, 8), (4, 0)])
def test_quantize_rows(loom, device, dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * 131 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(8 * torch.randn(rows, 1, generator=g)).clamp(1e-3, 1e3)
    check_quantize(loom, device, x.to(dtype).to(device))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("offset,pad", [(0, 4), (1, 3), (2, 6), (4, 0), (3, 5), (8, 8)])
def test_quantize_strided_and_unaligned(loom, device, dtype, offset, pad):
    for cols in (60, 1024, 5000):
        base = torch.randn(17 * (cols + pad) + offset, generator=torch.Generator().manual_seed(cols)).to(dtype).to(device)
        check_quantize(loom, device, base[offset:].as_strided((17, cols), (cols + pad, 1), offset))


def test_quantize_special_rows(loom, device):
    cols = 2052
    x = torch.randn(14, cols, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, 2051] = float("-inf")
    x[3, 0] = float("nan")
    x[4] = 1e-40                       # subnormal
    x[5] = 0
    x[5, 3] = TINY                     # the smallest live row
    x[6] = 0
    x[6, 3] = float(np.nextafter(np.float32(TINY), np.float32(0)))
    x[7] = 3.4028234663852886e38
    x[8] = torch.arange(cols) % 255 - 127.0   # exact integers, max 127
    x[9] = (torch.arange(cols) % 254 - 127) + 0.5  # halves: ties to even
    x[9, 0] = 127
    x[10, :] = -0.0
    x[11, -1] = 1e30
    x[12, 5], x[12, 6] = float("nan"), float("inf")
    check_quantize(loom, device, x.to(device))
    check_quantize(loom, device, x.to(BF16).to(device))
    # every value, and each place a lone infinity can sit in
    for c in list(range(0, 64)) + [255, 256, 511, 1023, 1024, 2047, 2048, 2051]:
        y = torch.zeros(2, cols)
        y[0, c], y[1, c] = float("nan"), -3.0
        check_quantize(loom, device, y.to(device))


# ------------------------------------------------------------------ the products

def operands(rows, k, tokens, seed, gated=False, device=None):
    g = torch.Generator().manual_seed(seed)
    s = {}
    for name in ("w", "u") if gated else ("w",):
        s[name] = torch.randint(-128, 128, (rows, k), generator=g, dtype=torch.int8)
        s[name + "s"] = (0.5 + torch.rand(rows, generator=g)) / (74 * 4 * max(1.0, math.sqrt(k)))
    s["x"] = torch.randint(-128, 128, (tokens, k), generator=g, dtype=torch.int8)
    s["xs"] = 0.02 + 0.08 * torch.rand(tokens, generator=g)
    s["bias"] = torch.randn(rows, generator=g)
    d = {n: (t if device is None else t.to(device)) for n, t in s.items()}
    return s, d


def accumulate(x, w):
    return (x.double() @ w.double().t()).to(torch.int64)  # |sums| < 2^31: exact


def scaled(acc, ws, xs):
    y = acc.float() * ws[None, :]  # int64 -> f32 is one rounding
    return y if xs is None else y * xs[:, None]


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


# channels, row length, tokens: around the tiles' edges, one of everything, rows that are not whole 16-byte chunks
SHAPES = [(1, 4, 1), (1, 8192, 1), (17, 20, 1), (64, 256, 3), (33, 1028, 16), (130, 64, 17), (16, 512, 2), (15, 252, 4),
          (48, 1024, 5), (100, 3328, 8), (257, 516, 65), (300, 1024, 130), (256, 2048, 64), (255, 132, 31),
          (512, 128, 256), (513, 192, 257), (129, 4096, 129), (1030, 320, 33), (77, 11008, 9), (2100, 260, 7),
          (640, 1024, 512), (31, 64, 1000), (384, 12, 300), (8, 16388, 12), (70, 131068, 3), (1500, 512, 700), (96, 0, 5)]


@pytest.mark.parametrize("rows,k,tokens", SHAPES)
def test_i8_matmul(loom, device, rows, k, tokens):
    s, d = operands(rows, k, tokens, rows + k + tokens, device=device)
    acc = accumulate(s["x"], s["w"])
    w, x = loom.pack_int8(d["w"]), loom.pack_int8(d["x"])
    for dtype in (F32, BF16, F16):
        want = (scaled(acc, s["ws"], s["xs"]) + s["bias"]).to(dtype)
        got = loom.i8_matmul(w, d["ws"], x, d["xs"], bias=d["bias"], dtype=dtype)
        assert same(got.cpu(), want), dtype
    assert same(loom.i8_matmul(w, d["ws"], x, dtype=F32).cpu(), scaled(acc, s["ws"], None))


def test_i8_matmul_limits(loom, device):
    """The accumulator's limits: all -128 against all -128 (2^31 - 2^16 at the longest row) and 127 against -128."""
    k = 131068
    for tokens in (1, 20, 70):
        for a, b in ((-128, -128), (127, -128)):
            w = torch.full((65, k), a, dtype=torch.int8, device=device)
            x = torch.full((tokens, k), b, dtype=torch.int8, device=device)
            got = loom.i8_matmul(loom.pack_int8(w), torch.ones(65, device=device), loom.pack_int8(x), dtype=F32)
            assert torch.all(got == float(np.float32(a * b * k)))


@pytest.mark.parametrize("tokens", [1, 3, 8, 16, 40, 64, 90, 128, 300])
def test_i8_matmul_one_hot(loom, device, tokens):
    """Each byte place of a row, one at a time, against distinct values: byte order, sign and every k position."""
    k = 320
    rows = k
    w = torch.eye(k, dtype=torch.int8)
    g = torch.Generator().manual_seed(tokens)
    x = torch.randint(-128, 128, (tokens, k), generator=g, dtype=torch.int8)
    one = torch.ones(rows, device=device)
    got = loom.i8_matmul(loom.pack_int8(w.to(device)), one, loom.pack_int8(x.to(device)), dtype=F32)
    assert torch.equal(got.cpu(), x.float())


def test_i8_matmul_views_and_scales(loom, device):
    """Operands that are only 4-byte aligned, strided outputs (whose gaps stay), special scales, a 1-d activation."""
    for rows, k, tokens in ((50, 1020, 3), (50, 1024, 3), (140, 1040, 40), (70, 256, 100), (300, 2048, 300)):
        s, d = operands(rows, k, tokens, 5, device=device)
        acc = accumulate(s["x"], s["w"])
        kw = k // 4
        for off in (0, 1, 2, 3):
            wb = torch.zeros(rows * kw + 8, dtype=torch.int32, device=device)
            xb = torch.zeros(tokens * kw + 8, dtype=torch.int32, device=device)
            w, x = wb[off:off + rows * kw].view(rows, kw), xb[off:off + tokens * kw].view(tokens, kw)
            w.copy_(loom.pack_int8(d["w"])), x.copy_(loom.pack_int8(d["x"]))
            for dtype in (F32, BF16):
                big = torch.full((tokens, rows + 5 + off), 7.0, dtype=dtype, device=device)
                out = big[:, 2 + off:2 + off + rows]
                assert loom.i8_matmul(w, d["ws"], x, d["xs"], out=out) is out
                want = torch.full(big.shape, 7.0, dtype=dtype)
                want[:, 2 + off:2 + off + rows] = scaled(acc, s["ws"], s["xs"]).to(dtype)
                assert torch.equal(big.cpu(), want)
        xs = s["xs"].clone()
        xs[0], xs[1], xs[2] = float("nan"), float("inf"), 0.0
        got = loom.i8_matmul(loom.pack_int8(d["w"]), d["ws"], loom.pack_int8(d["x"]), xs.to(device), dtype=F32).cpu()
        assert np.array_equal(got.numpy(), scaled(acc, s["ws"], xs).numpy(), equal_nan=True)
    one = loom.i8_matmul(loom.pack_int8(d["w"]), d["ws"], loom.pack_int8(d["x"])[0], dtype=F32)
    assert torch.equal(one.cpu(), scaled(acc[:1], s["ws"], None))


def act64(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if act == "relu":
        return g.clamp(min=0), (g > 0).double()
    if act == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)


def projections64(s):
    ag, au = accumulate(s["x"], s["w"]).double(), accumulate(s["x"], s["u"]).double()
    xs = s["xs"].double()[:, None]
    return ag * xs, au * xs, ag * s["ws"].double() * xs, au * s["us"].double() * xs


def within(got, want, tol):
    got = got.cpu().double()
    assert got.shape == want.shape
    over = (got - want).abs() - tol
    assert torch.isfinite(got).all() and (over <= 0).all(), (float(over.max()), float(want.abs().max()))


@pytest.mark.parametrize("rows,k,tokens", SHAPES)
def test_i8_gated_projection(loom, device, rows, k, tokens):
    s, d = operands(rows, k, tokens, 3 * rows + k + tokens, gated=True, device=device)
    s["ws"], d["ws"] = 4 * s["ws"], 4 * d["ws"]
    _, _, g, u = projections64(s)
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    for act in loom.ACTIVATIONS:
        a, _ = act64(g, act)
        for dtype in (F32, BF16, F16) if act == "silu" else (F32,):
            got = loom.i8_gated_projection(w, d["ws"], v, d["us"], x, d["xs"], act=act, dtype=dtype)
            assert got.dtype == dtype
            tol = (16 * g.abs() + 5 * a.abs()) * u.abs() * U
            within(got, a * u, tol + ((a * u).abs() + tol) * HALF[dtype] + LOW[dtype])


def test_i8_gated_projection_saturated(loom, device):
    """Gates far from 0 on both sides: no NaN, the limits 0 and g; scales that are 0, infinite and NaN propagate."""
    k = 64
    w = torch.ones(4, k, dtype=torch.int8, device=device)
    x = torch.tensor([[127] * k, [-128] * k, [0] * k], dtype=torch.int8, device=device)
    pw, px = loom.pack_int8(w), loom.pack_int8(x)
    gs = torch.tensor([1e-3, 1.0, 1e30, 0.0], device=device)
    one = torch.ones(4, device=device)
    for act in loom.ACTIVATIONS:
        got = loom.i8_gated_projection(pw, gs, pw, one, px, act=act, dtype=F32).cpu().double()
        g = (x.cpu().double().sum(1)[:, None] * gs.cpu().double()[None, :])
        a, _ = act64(g.clamp(-1e6, 1e38), act)
        u = x.cpu().double().sum(1)[:, None]
        within(got, a * u, (16 * g.abs() + 5 * a.abs()) * u.abs() * U + LOW[F32])
        assert not torch.isnan(got).any()
    bad = loom.i8_gated_projection(pw, torch.full((4,), float("nan"), device=device), pw, one, px, act="relu", dtype=F32)
    assert torch.isnan(bad).all()


# ------------------------------------------------------------------ gradients

def backward64(s, d_out, act):
    eg, eu, g, u = projections64(s)
    a, slope = act64(g, act)
    d = d_out.double()
    dg, du = d * u * slope, d * a
    ws, us = s["ws"].double(), s["us"].double()
    w, v = s["w"].double(), s["u"].double()
    d_x = (dg * ws) @ w + (du * us) @ v
    # the errors of dg and du in f32, and what they become
    eps_g = (d * u).abs() * (22 + 4 * g.abs()) * U
    eps_u = d.abs() * (16 * g.abs() + 6 * a.abs()) * U
    n = 2 * s["w"].shape[0]
    h = COEF[d_out.dtype]
    magnitude = (dg * ws).abs() @ w.abs() + (du * us).abs() @ v.abs()
    tol_x = (eps_g * ws) @ w.abs() + (eps_u * us) @ v.abs() + magnitude * (h + (6 + math.sqrt(n)) * U)
    tol_x = tol_x * (1 + HALF[d_out.dtype]) + d_x.abs() * HALF[d_out.dtype] + LOW[d_out.dtype]
    t = math.sqrt(s["x"].shape[0]) + 8
    tol_g = (eps_g * eg.abs()).sum(0) + (dg * eg).abs().sum(0) * t * U + LOW[F32]
    tol_u = (eps_u * eu.abs()).sum(0) + (du * eu).abs().sum(0) * t * U + LOW[F32]
    return (d_x, (dg * eg).sum(0), (du * eu).sum(0)), (tol_x, tol_g, tol_u)


@pytest.mark.parametrize("rows,k,tokens", [c for c in SHAPES if c[0] * c[1] * c[2] < 4e8])
def test_i8_gated_projection_backward(loom, device, rows, k, tokens):
    s, d = operands(rows, k, tokens, 5 * rows + k + tokens, gated=True, device=device)
    s["ws"], d["ws"] = 4 * s["ws"], 4 * d["ws"]
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    full = torch.randn(tokens, rows, generator=torch.Generator().manual_seed(k))
    for act in loom.ACTIVATIONS:
        for dtype in (F32, BF16, F16) if act == "silu" else (BF16,):
            d_out = full.to(dtype)
            want, tol = backward64(s, d_out, act)
            got = loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, d["xs"], d_out.to(device), act=act)
            assert got[0].dtype == dtype and got[1].dtype == got[2].dtype == F32
            for q, y, e in zip(got, want, tol):
                within(q, y, e)
    again = loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, d["xs"], d_out.to(device), act=act)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_oracle_gradients_against_differences():
    """The formulas of the gradients against central differences of the forward formula in float64."""
    s, _ = operands(6, 8, 5, 2, gated=True)
    s["ws"], s["us"] = 30 * s["ws"].double(), 30 * s["us"].double()
    s["xs"] = s["xs"].double()
    d_out = torch.randn(5, 6, dtype=torch.float64, generator=torch.Generator().manual_seed(3)).float()

    def loss(ws, us, xhat, act):
        g, u = xhat @ s["w"].double().t() * ws, xhat @ s["u"].double().t() * us
        return (act64(g, act)[0] * u * d_out.double()).sum()

    xhat = s["x"].double() * s["xs"][:, None]
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        (d_x, d_g, d_u), _ = backward64(s, d_out, act)
        for grad, which in ((d_g, 0), (d_u, 1), (d_x, 2)):
            args = [s["ws"], s["us"], xhat]
            for i in range(grad.numel()):
                e = torch.zeros_like(args[which]).view(-1)
                e[i] = 1e-5 * max(1e-3, float(args[which].view(-1)[i].abs()))
                e = e.view_as(args[which])
                hi = loss(*[a + e if j == which else a for j, a in enumerate(args)], act)
                lo = loss(*[a - e if j == which else a for j, a in enumerate(args)], act)
                slope = float(hi - lo) / (2 * float(e.abs().max()))
                assert abs(slope - float(grad.reshape(-1)[i])) <= 1e-4 * (abs(slope) + float(grad.abs().max())), (act, which, i)


def test_backward_against_differences_of_forward(loom, device):
    """The GPU's scale gradients against central differences of the GPU's f32 forward pass, along random directions."""
    s, d = operands(96, 512, 40, 8, gated=True, device=device)
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    ws, us = 8 * d["ws"], 8 * d["us"]
    d_out = torch.randn(40, 96, generator=torch.Generator().manual_seed(4)).to(device)
    _, dg, du = loom.i8_gated_projection_backward(w, ws, v, us, x, d["xs"], d_out, act="gelu")

    def loss(a, b):
        return float((loom.i8_gated_projection(w, a, v, b, x, d["xs"], act="gelu", dtype=F32).double() * d_out.double()).sum())

    for seed in range(3):
        r = torch.randn(96, generator=torch.Generator().manual_seed(seed)).to(device)
        h = 2.0 ** -7
        slope = (loss(ws * (1 + h * r), us) - loss(ws * (1 - h * r), us)) / (2 * h)
        want = float((dg.double() * ws.double() * r.double()).sum())
        size = float((dg.double() * ws.double() * r.double()).abs().sum())
        assert abs(slope - want) <= 1e-2 * size
        slope = (loss(ws, us * (1 + h * r)) - loss(ws, us * (1 - h * r))) / (2 * h)  # linear in up_scale
        want = float((du.double() * us.double() * r.double()).sum())
        assert abs(slope - want) <= 1e-4 * float((du.double() * us.double() * r.double()).abs().sum())


def test_backward_parts_and_empty(loom, device):
    s, d = operands(130, 260, 37, 4, gated=True, device=device)
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    big = torch.randn(37, 133, generator=torch.Generator().manual_seed(1)).to(BF16).to(device)
    d_out = big[:, 1:131]
    a = (w, d["ws"], v, d["us"], x, d["xs"], d_out)
    full = loom.i8_gated_projection_backward(*a)
    assert all(torch.equal(p, q) for p, q in zip(full, loom.i8_gated_projection_backward(*a[:-1], d_out.contiguous())))
    only_x = loom.i8_gated_projection_backward(*a, want_d_scales=False)
    only_s = loom.i8_gated_projection_backward(*a, want_d_x=False)
    assert torch.equal(only_x[0], full[0]) and only_x[1] is None and only_s[0] is None
    assert torch.equal(only_s[1], full[1]) and torch.equal(only_s[2], full[2])
    assert loom.i8_gated_projection_backward(*a, want_d_x=False, want_d_scales=False) == (None, None, None)
    # no tokens: zero scale gradients; no channels: a zero d_x
    none = loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x[:0], d["xs"][:0], d_out[:0].contiguous())
    assert tuple(none[0].shape) == (0, 260) and not none[1].any() and not none[2].any()
    none = loom.i8_gated_projection_backward(w[:0], d["ws"][:0], v[:0], d["us"][:0], x, d["xs"],
                                             torch.empty(37, 0, dtype=BF16, device=device))
    assert not none[0].any() and none[1].numel() == 0
    assert loom.i8_matmul(w[:0], d["ws"][:0], x, d["xs"]).shape == (37, 0)
    assert loom.i8_gated_projection(w, d["ws"], v, d["us"], x[:0], d["xs"][:0]).shape == (0, 130)


# ------------------------------------------------------------------ as a program uses them

def test_refusals(loom, device):
    s, d = operands(32, 64, 4, 1, gated=True, device=device)
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    d_out = torch.zeros(4, 32, device=device)
    for bad in (torch.zeros(2, 6, device=device), torch.zeros(8, device=device), torch.zeros(8, 8, device=device).t()):
        with pytest.raises(ValueError):
            loom.quantize_rows(bad[:, 1:] if bad.dim() == 2 and bad.stride(0) == 1 else bad)
    with pytest.raises(TypeError):
        loom.quantize_rows(torch.zeros(2, 8, dtype=torch.float64, device=device))
    with pytest.raises(ValueError):
        loom.quantize_rows(torch.zeros(2, 8, device=device).as_strided((2, 8), (4, 1)))
    refused = [lambda: loom.i8_matmul(w, d["ws"][:31], x, d["xs"]),
               lambda: loom.i8_matmul(w, d["ws"], x[:, :8], d["xs"]),
               lambda: loom.i8_matmul(w, d["ws"], x[:, :8].contiguous(), d["xs"]),
               lambda: loom.i8_matmul(w, d["ws"], x, d["xs"][:3]),
               lambda: loom.i8_matmul(w, d["ws"], x, d["xs"], bias=d["bias"][:31]),
               lambda: loom.i8_matmul(w, d["ws"], x, out=torch.zeros(32, 4, device=device)),
               lambda: loom.i8_matmul(w, d["ws"], x, out=torch.zeros(32, 4, device=device).t()),
               lambda: loom.i8_gated_projection(w, d["ws"], v[:31], d["us"], x),
               lambda: loom.i8_gated_projection(w, d["ws"], v, d["us"], x, act="tanh"),
               lambda: loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, None, d_out[:3]),
               lambda: loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, None, d_out,
                                                         workspace=torch.empty(8, dtype=torch.uint8, device=device))]
    for call in refused:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        loom.i8_matmul(w, d["ws"], x, dtype=torch.float64)
    with pytest.raises(TypeError):
        loom.i8_matmul(w.float(), d["ws"], x)
    with pytest.raises(TypeError):
        loom.i8_matmul(w, d["ws"].half(), x)
    need = loom.i8_gated_projection_backward_workspace(32, 64, 4, F32)
    off = torch.empty(need + 32, dtype=torch.uint8, device=device)[1:]
    with pytest.raises(loom.LoomError) as e:
        loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, None, d_out, workspace=off)
    assert e.value.status == loom.ERR_ALIGN


@pytest.mark.parametrize("tokens", [1, 12, 50, 300])
def test_streams_and_graph(loom, device, tokens):
    """A layer forward and its gradients on a side stream, then captured: every replay on new inputs gives the eager
    bits, with the program's own eager calls of the same operands between the replays."""
    rows, k = 520, 1040
    s, d = operands(rows, k, tokens, 6, gated=True, device=device)
    down = torch.randint(-128, 128, (k, rows), dtype=torch.int8, generator=torch.Generator().manual_seed(9)).to(device)
    ds = torch.rand(k, generator=torch.Generator().manual_seed(10)).to(device) / 500
    w, v, wd = loom.pack_int8(d["w"]), loom.pack_int8(d["u"]), loom.pack_int8(down)
    h = torch.randn(tokens, k, generator=torch.Generator().manual_seed(11)).to(BF16).to(device)

    def layer(h):
        q, qs = loom.quantize_rows(h)
        y = loom.i8_gated_projection(w, d["ws"], v, d["us"], q, qs)
        z, zs = loom.quantize_rows(y)
        out = loom.i8_matmul(wd, ds, z, zs)
        return (out, y) + loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], q, qs, y)

    want = [t.clone() for t in layer(h)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(h)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    static = h.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = layer(static)
    for step in range(4):
        h2 = (h.float() * (1 + step)).to(BF16).flip(0)
        eager = [t.clone() for t in layer(h2)]
        static.copy_(h2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), step


def test_offsets_past_32_bits(loom, device):
    """Weights past 2^31 bytes and outputs past 2^31 elements and 2^32 bytes."""
    k, rows = 131068, 17000  # 2.2 GB a weight
    w = torch.empty(rows, k // 4, dtype=torch.int32, device=device).random_(-2**31, 2**31 - 1)
    for tokens in (2, 40):
        x = torch.randint(-2**31, 2**31 - 1, (tokens, k // 4), dtype=torch.int32, device=device)
        got = loom.i8_matmul(w, torch.ones(rows, device=device), x, dtype=F32)
        tail = slice(rows - 40, rows)
        want = accumulate(x.cpu().view(torch.int8), w[tail].cpu().view(torch.int8)).float()
        assert torch.equal(got[:, tail].cpu(), want)
        d_out = torch.zeros(tokens, rows, device=device)
        d_out[:, tail] = 1.0
        one = torch.full((rows,), 1e-5, device=device)
        d_x, _, _ = loom.i8_gated_projection_backward(w, one, w, one, x, None, d_out)
        s = {"w": w[tail].cpu().view(torch.int8), "x": x.cpu().view(torch.int8), "ws": torch.full((40,), 1e-5),
             "us": torch.full((40,), 1e-5), "xs": torch.ones(tokens)}
        s["u"] = s["w"]
        (ref, _, _), (tol, _, _) = backward64(s, torch.ones(tokens, 40), "silu")
        within(d_x, ref, 3 * tol)  # the zero coefficients of the other channels add nothing
    del w, x, got, d_x
    tokens, rows, k = 70000, 32768, 4
    w = torch.randint(-2**31, 2**31 - 1, (rows, 1), dtype=torch.int32, device=device)
    x = torch.randint(-2**31, 2**31 - 1, (tokens, 1), dtype=torch.int32, device=device)
    got = loom.i8_matmul(w, torch.ones(rows, device=device), x, dtype=BF16)
    for part in (slice(0, 40), slice(65500, 65570), slice(tokens - 40, tokens)):
        want = accumulate(x[part].cpu().view(torch.int8), w.cpu().view(torch.int8)).float().to(BF16)
        assert torch.equal(got[part].cpu(), want)
    del got
    y = torch.randn(rows, 70000, device=device).to(BF16)
    q, scale = loom.quantize_rows(y)
    rq, rs = quantize_ref(y[-5:].cpu())
    assert np.array_equal(q[-5:].cpu().numpy().view(np.int8), rq) and np.array_equal(scale[-5:].cpu().numpy(), rs)
