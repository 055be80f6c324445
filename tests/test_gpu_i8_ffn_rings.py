"""Every tile shape of the int8 product, the gated projection and its gradients over rows of k that turn its rings of
LDS steps several times and end inside a step, with channels and tokens past a tile's edge.  SIZES names the shape that
each size takes; test_i8_ffn_shapes_cpu holds the library's launch geometry to it.

The product and the gated projection with ReLU are compared bit for bit: the int32 sums are exact and every f32 rounding
behind them is documented.  The gradients are held to the tolerances of test_gpu_i8_ffn."""
import pytest
import torch

from tests.test_gpu_i8_ffn import BF16, F32, backward64, operands, scaled

# (channels, tokens) of a tile of the product, waves, waves that split k, steps in the rings of weights and activations
TILES = [(32, 32, 2, 1, 5, 5), (64, 32, 4, 1, 6, 6), (64, 64, 4, 1, 5, 5), (128, 64, 4, 1, 3, 3), (64, 128, 4, 1, 3, 3),
         (128, 128, 4, 1, 5, 5), (128, 256, 4, 1, 4, 3), (256, 256, 4, 1, 2, 2), (32, 32, 4, 4, 4, 4), (32, 64, 4, 4, 3, 3)]

# operator -> {tile: sizes (channels, k, tokens)}; where a tile serves launches of one token tile, the last size is one
SIZES = {
    "i8_matmul": {
        0: [(33, 2052, 34), (33, 2052, 17)], 1: [(4302, 2052, 34), (8963, 2052, 17)],
        2: [(5495, 2052, 71), (8963, 2052, 34)], 3: [(11446, 1540, 71), (16517, 1540, 34)], 4: [(419, 1540, 4144)],
        5: [(11446, 2052, 129), (16517, 2052, 71)], 6: [(14616, 1540, 257), (23834, 1540, 129)],
        7: [(23834, 1540, 257)], 8: [(33, 8196, 34), (33, 8196, 17)], 9: [(33, 8196, 4144), (4302, 8196, 34)]},
    "i8_gated_projection": {
        0: [(33, 2052, 36), (33, 2052, 9)], 1: [(2065, 2052, 36), (4302, 2052, 9)],
        2: [(2981, 2052, 69), (4302, 2052, 36)], 3: [(3000, 1540, 165), (8963, 1540, 36)], 4: [(327, 1540, 2755)],
        5: [(5495, 2052, 139), (8963, 2052, 69)], 6: [(5495, 1540, 333), (11446, 1540, 139)],
        7: [(11446, 1540, 274), (16517, 1540, 139)], 8: [(33, 8196, 36), (33, 8196, 9)],
        9: [(33, 8196, 2755), (2065, 8196, 36)]},
    "i8_gated_projection_backward": {
        0: [(33, 2052, 36), (33, 2052, 9)], 1: [(2065, 2052, 36), (4302, 2052, 9)],
        2: [(2981, 2052, 69), (4302, 2052, 36)], 3: [(3000, 1540, 165), (8963, 1540, 36)], 4: [(327, 1540, 2755)],
        5: [(5495, 2052, 139), (8963, 2052, 69)], 6: [(5495, 1540, 333), (11446, 1540, 139)],
        7: [(11446, 1540, 274), (16517, 1540, 139)]},
}


def cases(op):
    return [pytest.param(*size, id=f"tile{tile}-" + "x".join(map(str, size)))
            for tile, sizes in SIZES[op].items() for size in sizes]


@pytest.fixture(scope="module")
def loom(device):
    import int8_dequant_dot_amd as m
    return m


def sums(x, w):
    return torch.mm(x.double(), w.double().t().contiguous()).to(torch.int64)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,tokens", cases("i8_matmul"))
def test_product(loom, device, rows, k, tokens):
    _, d = operands(rows, k, tokens, rows + k + tokens, device=device)
    want = scaled(sums(d["x"], d["w"]), d["ws"], d["xs"]) + d["bias"]
    w, x = loom.pack_int8(d["w"]), loom.pack_int8(d["x"])
    for dtype in (F32, BF16):
        got = loom.i8_matmul(w, d["ws"], x, d["xs"], bias=d["bias"], dtype=dtype)
        assert got.dtype == dtype and torch.equal(got, want.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,tokens", cases("i8_gated_projection"))
def test_gated(loom, device, rows, k, tokens):
    _, d = operands(rows, k, tokens, rows + k + tokens, gated=True, device=device)
    g, u = (scaled(sums(d["x"], d[n]), d[n + "s"], d["xs"]) for n in ("w", "u"))
    want = torch.where(g < 0, 0.0, g) * u
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    for dtype in (F32, BF16):
        got = loom.i8_gated_projection(w, d["ws"], v, d["us"], x, d["xs"], act="relu", dtype=dtype)
        assert got.dtype == dtype and torch.equal(got, want.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,tokens", cases("i8_gated_projection_backward"))
def test_gradients(loom, device, rows, k, tokens):
    _, d = operands(rows, k, tokens, rows + k + tokens, gated=True, device=device)
    d["ws"] = 4 * d["ws"]
    w, v, x = (loom.pack_int8(d[n]) for n in ("w", "u", "x"))
    d_out = torch.randn(tokens, rows, generator=torch.Generator().manual_seed(k)).to(device)
    for dtype in (F32, BF16):
        want, tol = backward64(d, d_out.to(dtype), "silu")
        got = loom.i8_gated_projection_backward(w, d["ws"], v, d["us"], x, d["xs"], d_out.to(dtype))
        for q, y, e in zip(got, want, tol):
            assert q.shape == y.shape and torch.isfinite(q).all()
            over = (q.double() - y).abs() - e
            assert (over <= 0).all(), (float(over.max()), float(y.abs().max()))
