"""The 4-bit products at sizes that run every kernel's main loop: each token count of the weight stream and each tile shape,
with one, two and four groups in 128 elements, over several steps of k and a rest, ragged in tokens and channels.

Which kernel a size takes is the launch table's choice; test_experts_tiles_cpu.py holds these sizes to it.  Tolerances are
those of test_gpu_experts.py."""
import pytest
import torch

from tests.test_gpu_experts import BF16, F16, F32, HALF, LOW, U, act64, bounded, loom, offsets_of, operands, parts  # noqa: F401

pytestmark = pytest.mark.gpu
K = 1312  # 5 steps of 256 (10 of 128) and a rest of 32

# (rows, tokens, group); routed: over 5 experts
DENSE = [(300, 2, 128), (300, 2, 64), (300, 7, 128), (300, 3, 64), (1120, 2, 32), (4099, 1000, 128), (4099, 1000, 64),
         (4099, 1000, 32), (2100, 1500, 128), (2100, 1500, 64), (2100, 1000, 32), (4099, 40, 128), (4099, 40, 64),
         (1541, 330, 32), (300, 11, 128), (300, 7, 64), (300, 3, 32)]
ROUTED = [(300, 2, 128), (300, 2, 64), (300, 2, 32), (4099, 1000, 128), (4099, 1000, 64), (4099, 1000, 32), (2100, 1500, 128),
          (2100, 1500, 64), (2100, 1000, 32), (2100, 40, 128), (4099, 11, 64), (4099, 7, 32), (300, 40, 128), (300, 11, 64),
          (300, 7, 32)]
GATED = [(300, 2, 128), (300, 2, 64), (300, 2, 32), (2100, 1000, 128), (2100, 1000, 64), (2100, 1000, 32), (1541, 330, 128),
         (1541, 330, 64), (2100, 330, 32), (4099, 40, 128), (4099, 11, 64), (4099, 129, 32), (300, 40, 128), (300, 11, 64),
         (300, 7, 32)]
EXPERTS = 5


def counts_of(pairs):
    """Rows of 5 experts: one has none, one a single row, one half of all; a few rows behind the last are left over."""
    left = min(3, pairs // 4)
    a, b = pairs // 2, min(1, pairs // 7)
    c = (pairs - left - a - b) // 3
    return [a, 0, b, c, pairs - left - a - b - c]


def product64(x, w, ws, group):
    """As there, computed where the operands are: (the sum, the sum of the parts' magnitudes)."""
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    size = y.clone()
    step = min(group, 128)
    for at in range(0, x.shape[1], step):
        part = slice(at, at + step)
        term = torch.mm(x[:, part].double(), w[:, part].double().t().contiguous()) * ws[:, at // group].double()
        y += term
        size += term.abs()
    return y, size


def held(got, v, tol):
    assert bool(((got.double() - v).abs() <= tol).all())


def on(device, s):
    return {n: t.to(device) for n, t in s.items()}


@pytest.mark.parametrize("rows,tokens,group", DENSE)
def test_dense(loom, device, rows, tokens, group):  # noqa: F811
    for dtype, scales in ((F32, F16), (BF16, F32)):
        d = on(device, operands(1, rows, K, tokens, group, scales, rows + tokens + group))
        y, size = product64(d["x"], d["w"][0], d["ws"][0], group)
        w, x = loom.pack_int4(d["w"][0]), loom.pack_int8(d["x"])
        big = torch.full((tokens, rows + 3), 7.0, dtype=dtype, device=device)
        loom.i4_matmul(w, d["ws"][0], x, d["xs"], bias=d["bias"][0], group=group, out=big[:, 1:1 + rows])
        held(big[:, 1:1 + rows], *bounded(y, size, parts(K, group), d["xs"], d["bias"][0], dtype))
        assert bool((big[:, :1] == 7).all()) and bool((big[:, 1 + rows:] == 7).all())


@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("rows,pairs,group", ROUTED)
def test_routed(loom, device, rows, pairs, group, indexed):  # noqa: F811
    offsets = offsets_of(counts_of(pairs))
    for dtype, scales in ((F32, BF16), (F16, F16)):
        d = on(device, operands(EXPERTS, rows, K, pairs, group, scales, rows + pairs + group))
        index = torch.randint(0, pairs, (pairs,), dtype=torch.int32, device=device) if indexed else None
        at = torch.arange(pairs, device=device) if index is None else index.long()
        out = torch.full((pairs, rows), 7.0, dtype=dtype, device=device)
        loom.i4_expert_matmul(loom.pack_int4(d["w"]), d["ws"], loom.pack_int8(d["x"]), d["xs"], offsets.to(device), index=index,
                              bias=d["bias"], group=group, out=out)
        for e, (a, b) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
            if a < b:
                y, size = product64(d["x"][at[a:b]], d["w"][e], d["ws"][e], group)
                held(out[a:b], *bounded(y, size, parts(K, group), d["xs"][at[a:b]], d["bias"][e], dtype))
        assert bool((out[int(offsets[-1]):] == 7).all())


@pytest.mark.parametrize("rows,pairs,group", GATED)
def test_gated(loom, device, rows, pairs, group):  # noqa: F811
    offsets = offsets_of(counts_of(pairs))
    for dtype, scales, act in ((F32, F16, "silu"), (BF16, F32, "gelu_tanh")):
        d = on(device, operands(EXPERTS, rows, K, pairs, group, scales, rows + pairs + group, ("w", "u")))
        index = torch.randint(0, pairs, (pairs,), dtype=torch.int32, device=device)
        at = index.long()
        out = torch.full((pairs, rows), 7.0, dtype=dtype, device=device)
        loom.i4_expert_gated_projection(loom.pack_int4(d["w"]), d["ws"], loom.pack_int4(d["u"]), d["us"], loom.pack_int8(d["x"]),
                                        d["xs"], offsets.to(device), index=index, act=act, group=group, out=out)
        for e, (a, b) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
            if a == b:
                continue
            x, xs, n = d["x"][at[a:b]], d["xs"][at[a:b]], parts(K, group)
            gv, gt = bounded(*product64(x, d["w"][e], d["ws"][e], group), n, xs, None, F32)
            uv, ut = bounded(*product64(x, d["u"][e], d["us"][e], group), n, xs, None, F32)
            v = act64(gv, act) * uv
            # |act'| <= 1.13; act itself within (16 |g| + 5 |act|) u
            tol = (1.13 * gt + (16 * gv.abs() + 5 * act64(gv, act).abs()) * U) * (uv.abs() + ut) + act64(gv, act).abs() * ut
            held(out[a:b], v, tol * (1 + HALF[dtype]) + (HALF[dtype] + U) * v.abs() + LOW[dtype])
        assert bool((out[int(offsets[-1]):] == 7).all())


@pytest.mark.parametrize("rows,tokens,group", [(4099, 1000, 128), (2100, 1500, 64), (4099, 1000, 32)])
def test_large_tiles_same_bits(loom, device, rows, tokens, group):  # noqa: F811
    """Tiles whose waves meet at every step: the same bits on every call, on two streams at once and in a graph's replays."""
    d = on(device, operands(EXPERTS, rows, K, tokens, group, F16, 5, ("w", "u")))
    w, u, x = loom.pack_int4(d["w"]), loom.pack_int4(d["u"]), loom.pack_int8(d["x"])
    offsets = offsets_of(counts_of(tokens)).to(device)

    def run():
        out = torch.zeros(2, tokens, rows, device=device)
        loom.i4_expert_matmul(w, d["ws"], x, d["xs"], offsets, group=group, out=out[0])
        loom.i4_expert_gated_projection(w, d["ws"], u, d["us"], x, d["xs"], offsets, group=group, out=out[1])
        return loom.i4_matmul(w[0], d["ws"][0], x, d["xs"], group=group, dtype=F32), out

    want = run()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(2):
        for stream in streams:
            with torch.cuda.stream(stream):
                got.append(run())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(want, r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
