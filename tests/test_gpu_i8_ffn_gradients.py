"""The gated projection's gradients in bfloat16: the accuracy of d_x and the range of its coefficients, in float32 and
float16 where they share it.

Tolerances: those of test_gpu_i8_ffn, with the coefficients of bfloat16 gradients rounded to 11 bits (half a step: 2^-11
of each, and no less than 2^-30 of the token's largest, below which they run out of exponents)."""
import math

import pytest
import torch

from tests.test_gpu_i8_ffn import BF16, COEF, F16, F32, HALF, act64, backward64, operands, projections64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


def gradients(loom, d, d_out):
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    return loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, d["xs"], d_out)


def coefficients64(d, d_out, act="silu"):
    """dg * gate_scale and du * up_scale in float64."""
    _, _, g, u = projections64(d)
    a, slope = act64(g, act)
    t = d_out.double()
    return t * u * slope * d["ws"].double(), t * a * d["us"].double()


def near(got, want, tol):
    assert got.shape == want.shape and torch.isfinite(got).all()
    over = (got.double() - want).abs() - tol
    assert (over <= 0).all(), (float(over.max()), float(want.abs().max()))


@pytest.mark.parametrize("rows,k,tokens", [(700, 516, 65), (2052, 132, 257), (4100, 1028, 300), (3000, 2052, 9), (700, 4100, 952)])
def test_bfloat16_d_x_is_rounded_once(loom, device, rows, k, tokens):
    """d_x in bfloat16 is as far from the exact gradient as the exact gradient rounded to bfloat16, but for what 11 bits of
    the coefficients leave: independent errors of at most 2^-11 of each term, a standard deviation of at most 2^-11 times
    the root of the sum of the terms' squares.  5 % is for the statistics of some 10^4 values and more."""
    _, d = operands(rows, k, tokens, rows + k + tokens, gated=True, device=device)
    d["ws"] = 4 * d["ws"]
    d_out = torch.randn(tokens, rows, generator=torch.Generator().manual_seed(k)).to(BF16).to(device)
    cg, cu = coefficients64(d, d_out)
    w, v = d["w"].double(), d["u"].double()
    want = cg @ w + cu @ v
    terms = (cg.square() @ w.square() + cu.square() @ v.square()).mean()
    rounded = (want.to(BF16).double() - want).square().mean()
    got = gradients(loom, d, d_out)[0]
    off = (got.double() - want).square().mean()
    assert off.sqrt() <= 1.05 * (rounded + 2.0 ** -22 * terms).sqrt(), (float(off.sqrt()), float(rounded.sqrt()))


def blocks_of(rows, tokens, seed):
    """Powers of two for each token and group of 16 channels, far apart."""
    g = torch.Generator().manual_seed(seed)
    groups = -(-rows // 16)
    low = 2.0 ** torch.randint(-36, 1, (tokens, groups), generator=g)
    return (2.0 ** torch.randint(-30, 31, (tokens, 1), generator=g) * low).repeat_interleave(16, 1)[:, :rows]


@pytest.mark.parametrize("rows,k,tokens", [(40, 68, 9), (700, 132, 12), (2065, 132, 36), (2981, 260, 69), (5495, 132, 139),
                                           (11446, 132, 274), (1000, 516, 1025)])
def test_bfloat16_coefficients_of_any_size(loom, device, rows, k, tokens):
    """Gradients whose channels differ by up to 2^36 within a token and tokens by 2^60, a token without any, and one whose
    gradients are only in its last channel."""
    _, d = operands(rows, k, tokens, rows + tokens, gated=True, device=device)
    d["ws"] = 4 * d["ws"]
    full = torch.randn(tokens, rows, generator=torch.Generator().manual_seed(k)) * blocks_of(rows, tokens, k)
    full[3], full[5, :-1] = 0, 0
    d_out = full.to(BF16).to(device)
    (want, want_g, want_u), (tol, tol_g, tol_u) = backward64(d, d_out, "silu")
    cg, cu = coefficients64(d, d_out)
    w, v = d["w"].double().abs(), d["u"].double().abs()
    # backward64's tolerance with the coefficients' 2^-8 replaced
    magnitude = cg.abs() @ w + cu.abs() @ v
    top = torch.maximum(cg.abs().amax(1), cu.abs().amax(1))[:, None]
    tol = tol + (1 + HALF[BF16]) * (magnitude * (2.0 ** -11 - COEF[BF16]) + 2.0 ** -30 * top * (w.sum(0) + v.sum(0)))
    got = gradients(loom, d, d_out)
    near(got[0], want, tol)
    near(got[1], want_g, tol_g)
    near(got[2], want_u, tol_u)
    assert not got[0][3].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_powers_of_two_pass_through(loom, device, dtype):
    """d_out times 2^24 or 2^-24 gives every gradient times the same, to the bit."""
    _, d = operands(700, 516, 70, 11, gated=True, device=device)
    d_out = torch.randn(70, 700, generator=torch.Generator().manual_seed(2)).to(dtype).to(device)
    base = gradients(loom, d, d_out)
    for power in (24, -24):
        got = gradients(loom, d, d_out * 2.0 ** power)
        assert all(torch.equal(a, b * 2.0 ** power) for a, b in zip(got, base))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_infinite_coefficients(loom, device, dtype):
    """An infinite gradient of one channel: plus or minus infinity where the channel's weight is not 0, NaN where it is,
    and other tokens keep their bits."""
    _, d = operands(300, 132, 20, 7, gated=True, device=device)
    d_out = torch.randn(20, 300, generator=torch.Generator().manual_seed(3)).to(dtype).to(device)
    clean = gradients(loom, d, d_out)[0]
    d_out[4, 9], d_out[11, 299], d_out[12, 0], d_out[12, 299] = math.inf, -math.inf, math.inf, -math.inf
    got = gradients(loom, d, d_out)[0]
    cg, cu = coefficients64(d, d_out)
    want = cg.cpu() @ d["w"].double().cpu() + cu.cpu() @ d["u"].double().cpu()
    for t in range(20):
        if t in (4, 11, 12):
            assert torch.equal(got[t].cpu().double().nan_to_num(7.0, 1.0, -1.0), want[t].nan_to_num(7.0, 1.0, -1.0))
        else:
            assert torch.equal(got[t], clean[t])
