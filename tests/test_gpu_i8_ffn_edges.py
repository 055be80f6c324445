"""The gated projection's gradients at the edges of their sizes: d_out that is unaligned or strided, coefficients past 2^31
elements, channels up to their limit.  Tolerances are those of test_gpu_i8_ffn."""
import math

import pytest
import torch

from tests.test_gpu_i8_ffn import BF16, F16, F32, backward64, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


def gradients(loom, d, d_out):
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    return loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, d["xs"], d_out)


def near(got, want, tol):
    assert got.shape == want.shape and torch.isfinite(got).all()
    over = (got.double() - want).abs() - tol
    assert (over <= 0).all(), (float(over.max()), float(want.abs().max()))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (2, 3), (3, 1), (4, 4), (5, 7)])
def test_d_out_of_any_alignment_and_stride(loom, device, dtype, offset, pad):
    for rows, k, tokens in ((130, 260, 37), (4100, 132, 9), (333, 132, 300)):
        _, d = operands(rows, k, tokens, rows, gated=True, device=device)
        base = torch.randn(tokens * (rows + pad) + offset, generator=torch.Generator().manual_seed(offset)).to(dtype).to(device)
        d_out = base.as_strided((tokens, rows), (rows + pad, 1), offset)
        want = gradients(loom, d, d_out.clone())
        got = gradients(loom, d, d_out)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ref, tol = backward64(d, d_out, "silu")
        for g, y, e in zip(got, ref, tol):
            near(g, y, e)


@pytest.mark.parametrize("dtype,rows,k,tokens", [(BF16, 28672, 64, 40000), (F32, 28672, 68, 12600)])
def test_coefficients_past_2_31_elements(loom, device, dtype, rows, k, tokens):
    """Limbs x tokens x 2 x channels past 2^31; d_x of the first tokens, the last, and those round that place."""
    g = torch.Generator(device=device).manual_seed(1)
    _, d = operands(rows, k, 1, 9, gated=True, device=device)
    d["x"] = torch.randint(-128, 128, (tokens, k), generator=g, dtype=torch.int8, device=device)
    d["xs"] = 0.02 + 0.08 * torch.rand(tokens, generator=g, device=device)
    d_out = torch.randn(tokens, rows, generator=g, dtype=F32, device=device).to(dtype)
    got = gradients(loom, d, d_out)
    at = 2 ** 31 // (2 * rows)
    for a, b in ((0, 40), (tokens - 40, tokens), (min(at, tokens) - 40, min(at + 40, tokens))):
        s = dict(d, x=d["x"][a:b], xs=d["xs"][a:b])
        (want, _, _), (tol, _, _) = backward64(s, d_out[a:b], "silu")
        near(got[0][a:b], want, tol)
    want_g, want_u, tol_g, tol_u = 0, 0, 0, 0
    for a in range(0, tokens, 2000):
        s = dict(d, x=d["x"][a:a + 2000], xs=d["xs"][a:a + 2000])
        (_, dg, du), (_, eg, eu) = backward64(s, d_out[a:a + 2000], "silu")
        want_g, want_u, tol_g, tol_u = want_g + dg, want_u + du, tol_g + eg, tol_u + eu
    # the chunks' tolerances hold the terms' and sqrt(2000) + 8 roundings of the sums: sqrt(tokens) + 8 are at most 5 times that
    near(got[1], want_g, 5 * tol_g)
    near(got[2], want_u, 5 * tol_u)


@pytest.mark.parametrize("dtype,rows,k,tokens", [(BF16, 2 ** 21, 256, 260), (BF16, 2 ** 20 + 70, 132, 33),
                                                 (F16, 2 ** 20 + 70, 68, 70), (F32, 2 ** 21 - 3, 68, 40)])
def test_channels_up_to_their_limit(loom, device, dtype, rows, k, tokens):
    """More than 2^20 channels, up to the 2^21 that the gradients take."""
    g = torch.Generator(device=device).manual_seed(1)
    d = {n: torch.randint(-128, 128, (r, k), generator=g, dtype=torch.int8, device=device)
         for n, r in (("w", rows), ("u", rows), ("x", tokens))}
    d["ws"], d["us"] = ((0.5 + torch.rand(rows, generator=g, device=device)) / (74 * 4 * math.sqrt(k)) for _ in range(2))
    d["xs"] = 0.02 + 0.08 * torch.rand(tokens, generator=g, device=device)
    d_out = torch.randn(tokens, rows, generator=g, dtype=F32, device=device).to(dtype)
    got = gradients(loom, d, d_out)
    want, tol = [0, [], []], [0, [], []]
    parts = range(0, rows, 2 ** 18)
    for a in parts:
        s = dict(d, **{n: d[n][a:a + 2 ** 18] for n in ("w", "u", "ws", "us")})
        values, errors = backward64(s, d_out[:, a:a + 2 ** 18], "silu")
        want[0], tol[0] = want[0] + values[0], tol[0] + errors[0]
        for i in (1, 2):
            want[i].append(values[i])
            tol[i].append(errors[i])
    # a chunk's sums of n terms have (6 + sqrt(n)) roundings, the whole's sqrt(chunks) times that
    near(got[0], want[0], math.sqrt(len(parts)) * tol[0])
    for i in (1, 2):
        near(got[i], torch.cat(want[i]), torch.cat(tol[i]))
