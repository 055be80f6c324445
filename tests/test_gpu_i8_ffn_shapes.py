"""The int8 feed-forward operators at sizes that take each of their tile shapes, against float64 on the GPU, and the
layer of the example.  Tolerances are those of test_gpu_i8_ffn."""
import importlib.util
import os

import pytest
import torch

from tests.test_gpu_i8_ffn import BF16, COEF, F16, F32, HALF, LOW, U, act64, backward64, operands, projections64, scaled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


# (channels, k, tokens) that reach tiles of 32 x 32, 64 x 32, 64 x 64, 128 x 64, 64 x 128, 128 x 128, 128 x 256 and
# 256 x 256 (channels x tokens) for the product or the gated projection, and of 32 x 32 whose waves split k, most with
# one whole step of k and one that is partly filled (test_gpu_i8_ffn_rings: every tile of each operator, longer rows)
SIZES = [(33, 132, 17), (500, 4100, 21), (500, 4100, 60), (100, 128, 33), (100, 60, 20), (33, 132, 4100), (8200, 132, 33), (16400, 132, 33), (4096, 1024, 512), (16400, 132, 65),
         (16400, 132, 200), (16400, 132, 257), (33, 132, 9), (4100, 132, 9), (4100, 132, 33), (16400, 132, 9),
         (200, 132, 4100), (8200, 132, 65), (11000, 132, 129), (2048, 2176, 2048)]


def near(got, want, tol):
    assert got.shape == want.shape and torch.isfinite(got).all()
    over = (got.double() - want).abs() - tol
    assert (over <= 0).all(), (float(over.max()), float(want.abs().max()))


@pytest.mark.parametrize("rows,k,tokens", SIZES)
def test_product_and_gated_shapes(loom, device, rows, k, tokens):
    _, d = operands(rows, k, tokens, rows + 7 * k + tokens, gated=True, device=device)
    w, u, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    acc = torch.mm(d["x"].double(), d["w"].double().t().contiguous()).to(torch.int64)
    want = scaled(acc, d["ws"], d["xs"]) + d["bias"]
    for dtype in (F32, BF16):
        got = loom.i8_matmul(w, d["ws"], x, d["xs"], bias=d["bias"], dtype=dtype)
        assert got.dtype == dtype and torch.equal(got, want.to(dtype))
    d["ws"] = 4 * d["ws"]
    _, _, g, up = projections64(d)
    for act, dtype in (("silu", BF16), ("gelu", F32), ("gelu_tanh", F16)):
        a, _ = act64(g, act)
        tol = (16 * g.abs() + 5 * a.abs()) * up.abs() * U
        got = loom.i8_gated_projection(w, d["ws"], u, d["us"], x, d["xs"], act=act, dtype=dtype)
        assert got.dtype == dtype
        near(got, a * up, tol + ((a * up).abs() + tol) * HALF[dtype] + LOW[dtype])


# d_x in tiles of 256 x 256, 128 x 128, 128 x 32 and 256 x 128 (columns x tokens), whole and in a few or many parts
@pytest.mark.parametrize("dtype,rows,k,tokens", [
    (BF16, 33, 2052, 4100), (BF16, 4100, 4100, 1025), (BF16, 33, 132, 4100), (BF16, 1500, 132, 1025),
    (BF16, 6000, 132, 200), (BF16, 700, 132, 9), (BF16, 2052, 132, 9), (BF16, 33, 4100, 1025), (BF16, 2052, 4100, 129),
    (BF16, 3000, 4100, 33), (F32, 33, 2052, 1025), (F32, 700, 132, 4100), (F32, 4100, 132, 700), (F32, 2052, 132, 9),
    (F32, 33, 4100, 1025), (F32, 3000, 132, 4100), (F32, 4100, 4100, 65), (F16, 33, 2052, 1025), (F16, 1500, 132, 1500),
    (F16, 700, 132, 9), (F16, 33, 4100, 1025), (F16, 4100, 4100, 65)])
def test_backward_shapes(loom, device, dtype, rows, k, tokens):
    _, d = operands(rows, k, tokens, rows + k + 3 * tokens, gated=True, device=device)
    d["ws"] = 4 * d["ws"]
    w, u, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    d_out = torch.randn(tokens, rows, generator=torch.Generator().manual_seed(k)).to(dtype).to(device)
    assert COEF[dtype] > 0
    want, tol = backward64(d, d_out, "silu")
    got = loom.i8_gated_projection_backward(w, d["ws"], u, d["us"], x, d["xs"], d_out)
    for g, y, e in zip(got, want, tol):
        near(g, y, e)
    again = loom.i8_gated_projection_backward(w, d["ws"], u, d["us"], x, d["xs"], d_out)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_special_values(loom, device):
    """A token whose scale is NaN or infinite stays its own: other tokens' gradients keep their bits; channels whose
    gradient of the output is infinite make that token's d_x infinite or NaN, nobody else's."""
    _, d = operands(200, 516, 40, 3, gated=True, device=device)
    w, u, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    for dtype in (F32, F16, BF16):
        d_out = torch.randn(40, 200, generator=torch.Generator().manual_seed(1)).to(dtype).to(device)
        clean = loom.i8_gated_projection_backward(w, d["ws"], u, d["us"], x, d["xs"], d_out)[0]
        xs, bad = d["xs"].clone(), d_out.clone()
        xs[3], xs[17] = float("nan"), float("inf")
        bad[31, 7] = float("inf")
        got = loom.i8_gated_projection_backward(w, d["ws"], u, d["us"], x, xs, bad)[0]
        rest = [t for t in range(40) if t not in (3, 17, 31)]
        assert torch.equal(got[rest], clean[rest])
        for t in (3, 17, 31):
            assert not torch.isfinite(got[t]).all()


def test_backward_row_limit(loom, device):
    """More channels than the gradients take are refused before anything is launched."""
    with pytest.raises(loom.LoomError) as e:
        loom.i8_gated_projection_backward_workspace(2 ** 21 + 1, 64, 4)
    assert e.value.status == loom.ERR_RANGE


def test_example_layer(loom, device):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_feed_forward.py")
    spec = importlib.util.spec_from_file_location("int8_feed_forward", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for tokens in (1, 96):
        error, losses = example.main(hidden=512, inner=1376, tokens=tokens, steps=5)
        # each of the four roundings to int8 is off by at most half a step of the row's 1/127, about 1 % of its typical value
        assert error < 0.05
        assert losses[-1] < losses[0]
