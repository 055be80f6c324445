"""Where the router's f32 choices and the 4-bit products come to their ends: groups whose values nearly tie, biases of the
lowest value, infinite and vanishing scales, offsets that overlap.  Against 64-bit values, tolerances as in
test_gpu_experts.py."""
import pytest
import torch

from tests.test_gpu_experts import (BF16, F16, F32, INF, bounded, check, check_route, loom, offsets_of,  # noqa: F401
                                    operands, parts, product64)

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(F32).min


# ------------------------------------------------------------------ groups that nearly tie

def best_of_two_groups(logits, bias):
    """The two experts of the better of two groups of two, falling, from 64-bit choices (sigmoid and bias)."""
    c = torch.sigmoid(logits.double()) + bias.double()
    first = (c[:, 2] + c[:, 3]) > (c[:, 0] + c[:, 1])
    ids = torch.empty(len(logits), 2, dtype=torch.int32)
    for g in (0, 1):
        pair = torch.where((c[:, 2 * g + 1] > c[:, 2 * g])[:, None], torch.tensor([2 * g + 1, 2 * g]), torch.tensor([2 * g, 2 * g + 1]))
        ids[first == bool(g)] = pair.to(torch.int32)[first == bool(g)]
    return ids


def check_groups(loom, device, logits, bias):  # noqa: F811
    """As groups of two, and as groups of eight whose other experts are masked; as a batch, and a few tokens at a time."""
    want = best_of_two_groups(logits, bias)
    wide, wide_bias = torch.full((len(logits), 16), -INF), torch.zeros(16)
    at = torch.tensor([1, 6, 10, 13])
    wide[:, at], wide_bias[at] = logits, bias
    for few in (False, True):
        def ids(l, b):
            l, b = l.to(device), b.to(device)
            runs = l.split(600) if few else [l]
            return torch.cat([loom.route_experts(r, 2, "sigmoid", b, 2, 1, 2)[0] for r in runs]).cpu()
        assert torch.equal(ids(logits, bias), want)
        assert torch.equal(ids(wide, wide_bias), at.to(torch.int32)[want.long()])


@pytest.mark.parametrize("step", [2.0 ** -21, 2.0 ** -20, 2.0 ** -19])
def test_groups_near_half_steps(loom, device, step):  # noqa: F811
    """Choices next to half steps of f32, in sums that round in opposite directions: the worst of f32 for two groups."""
    c = step * 2.0 ** 23 + (torch.tensor([1001, 2000, 1600, 1401], dtype=torch.float64) + 0.5) * step
    near = c - 0.8 + 0.005 * torch.arange(4)
    bias = (near / (step / 2)).round() * (step / 2)  # held exactly
    l = torch.logit(c - bias).float()
    j = torch.arange(-6, 7)
    grid = torch.cartesian_prod(j, j, j, j)
    logits = (l.view(torch.int32)[None] + grid.to(torch.int32)).view(F32).contiguous()
    check_groups(loom, device, logits, bias.float())
    swap = torch.tensor([2, 3, 0, 1])
    check_groups(loom, device, logits[:, swap].contiguous(), bias.float()[swap])


@pytest.mark.parametrize("size", [0.25, 7.0, 100.0, 1000.0, 30000.0])
def test_groups_near_ties(loom, device, size):  # noqa: F811
    """Random tokens whose second group is moved to within a few steps of the first."""
    g = torch.Generator().manual_seed(int(size))
    bias = size * (1 + 1e-4 * torch.rand(4, generator=g))
    bias[3] = (bias[0].double() + bias[1].double() - bias[2].double()).float()
    s = 0.3 + 0.4 * torch.rand(20000, 4, generator=g, dtype=torch.float64)
    b = bias.double()
    s[:, 3] = s[:, 0] + s[:, 1] - s[:, 2] + (b[0] + b[1] - b[2] - b[3])
    s = s[(s[:, 3] > 0.05) & (s[:, 3] < 0.95)]
    logits = torch.logit(s).float()
    logits[:, 3] = (logits[:, 3].view(torch.int32) + torch.randint(-8, 9, (len(s),), generator=g, dtype=torch.int32)).view(F32)
    assert len(s) > 5000
    check_groups(loom, device, logits, bias)


def test_groups_one_token(loom, device):  # noqa: F811
    """Second group ahead by 2.2e-7, the first by 3.8e-6 if every step is rounded to f32."""
    logits = torch.tensor([[float.fromhex(v) for v in ("0x1.731936p0", "0x1.697162p0", "0x1.6cb4c4p0", "0x1.700cf4p0")]])
    bias = torch.tensor([7.19006395, 7.19593716, 7.19393682, 7.19190359])
    check_groups(loom, device, logits, bias)


# ------------------------------------------------------------------ biases of the lowest value

@pytest.mark.parametrize("tokens", [9, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_lowest_biases(loom, device, score, tokens):  # noqa: F811
    """Groups whose two best choices add up to less than the lowest f32 value are groups all the same: better than those
    whose experts are all masked, in the order of their 64-bit sums."""
    for size, kept in ((2, 3), (8, 3), (8, 5)):
        experts = 6 * size
        g = torch.Generator().manual_seed(size)
        logits = torch.randn(tokens, experts, generator=g)
        logits[:, :size] = -INF                        # group 0: nothing
        bias = torch.zeros(experts)
        bias[size:2 * size] = LOWEST                   # 1: the lowest value throughout
        bias[2 * size:3 * size] = -2.5e38              # 2: lower sum than 3
        bias[3 * size:4 * size] = -2.0e38
        bias[4 * size:5 * size] = LOWEST               # 4: one expert is not
        bias[4 * size] = 0.5
        bias[5 * size] = LOWEST                        # 5: one expert is
        check_route(loom, device, logits.to(device), 3, score, bias, 6, kept, 2)
        check_route(loom, device, logits.to(device), 2 * size, score, bias, 6, kept, 2, False)
        check_route(loom, device, logits.to(device), min(3, size), score, -bias, 6, 1, 2)  # and sums beyond the largest
        check_route(loom, device, logits.to(device), 3, score, -bias, 6, kept, 2)


@pytest.mark.parametrize("tokens", [9, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_lowest_biases_beside_small_ones(loom, device, score, tokens):  # noqa: F811
    """A few experts shut by the lowest value, the others ordered by ordinary biases, with near ties among them; large
    biases apart from small ones; tokens without any expert between the others."""
    experts = 64
    g = torch.Generator().manual_seed(21)
    logits = (1 + torch.randint(0, 40, (tokens, experts), generator=g) * 2.0 ** -23).float()
    logits[::3] = torch.randn(len(logits[::3]), experts, generator=g)
    logits[4::7] = -INF
    bias = 0.1 * torch.randn(experts, generator=g)
    bias[8:16] = bias[:8]
    bias[[0, 17, 40]] = LOWEST
    bias[[1, 41]] = -1e9
    bias[2] = 1e4
    for groups, kept, top_group in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (32, 9, 2)):
        check_route(loom, device, logits.to(device), 8, score, bias, groups, kept, top_group)
        check_route(loom, device, logits.to(device), 8, score, bias, groups, kept, top_group, False)


# ------------------------------------------------------------------ many choices

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top_k", [11, 12, 13, 14, 15, 16, 17])
def test_many_choices(loom, device, top_k, score):  # noqa: F811
    """Batches in which a token's lanes are nearly all taken by its choices, ties and near ties among them."""
    g = torch.Generator().manual_seed(top_k)
    logits = torch.randn(1030, 48, generator=g)
    logits[::5] = (1 + torch.randint(0, 3, (len(logits[::5]), 48), generator=g) * 2.0 ** -23).float()
    bias = torch.zeros(48)
    bias[::3] = 2.0 ** -26
    for groups, kept in ((1, 1), (4, 2)):
        for dtype in (F32, BF16, F16):
            check_route(loom, device, logits.to(dtype).to(device), top_k, score, bias, groups, kept)
            check_route(loom, device, logits.to(dtype).to(device), top_k, score, None, groups, kept, 1, False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k", [(130, 64, 64), (130, 65, 64), (130, 63, 63), (130, 200, 63), (130, 200, 64),
                                                  (40, 1000, 64), (1030, 16, 16), (1030, 17, 16), (1030, 250, 16)])
def test_every_lane_a_choice(loom, device, tokens, experts, top_k, score):  # noqa: F811
    """As many choices as a token has lanes: one more is looked at, where there is one, and rows with fewer experts end
    before it."""
    g = torch.Generator().manual_seed(experts)
    logits = torch.randn(tokens, experts, generator=g)
    logits[1::4] = (1 + torch.randint(0, 3, (len(logits[1::4]), experts), generator=g) * 2.0 ** -23).float()
    logits[2::9, top_k - 1:] = -INF
    logits[3::9, 5:] = -INF
    logits[4::9] = -INF
    bias = 0.1 * torch.randn(experts, generator=g)
    for dtype in (F32, BF16):
        check_route(loom, device, logits.to(dtype).to(device), top_k, score, bias)
        check_route(loom, device, logits.to(dtype).to(device), top_k, score, None, renormalize=False)


# ------------------------------------------------------------------ scales at the ends of their range

SIZES = [(70, 1056, 32), (70, 544, 32), (70, 1056, 64), (70, 544, 64), (70, 32, 32), (70, 1056, 128), (70, 672, 128),
         (70, 2080, 256), (40, 4192, 512)]


@pytest.mark.parametrize("tokens", [1, 2, 3, 7, 8, 9, 40, 300])
@pytest.mark.parametrize("rows,k,group", SIZES)
def test_infinite_scales(loom, device, rows, k, group, tokens):  # noqa: F811
    """An infinite scale of a row's last group makes its channel infinite, of the sign that the group's sum has; no other
    channel sees it.  The same at every token count.  (The last groups here are at most 128 long: longer ones are added in
    parts, which may be infinite in both directions.)"""
    for scales in (F32, F16):
        s = operands(2, rows, k, tokens, group, scales, rows + k + tokens)
        last = slice((k - 1) // group * group, k)
        s["w"][:, :, last] = s["w"][:, :, last].abs() + 1
        s["x"][:, last] = s["x"][:, last].clamp(-127, 127).abs() + (s["x"][:, last] == 0)
        s["w"].clamp_(-8, 7)
        s["ws"][:, 3, -1], s["ws"][:, 64 if rows > 64 else 33, -1] = INF, -INF
        want = torch.zeros(rows)
        want[3], want[64 if rows > 64 else 33] = INF, -INF
        other = want == 0
        d = {n: t.to(device) for n, t in s.items()}
        w, x = loom.pack_int4(d["w"]), loom.pack_int8(d["x"])
        got = [loom.i4_matmul(w[1], d["ws"][1], x, group=group, dtype=F32).cpu(),
               loom.i4_expert_matmul(w, d["ws"], x, None, offsets_of([0, tokens]).to(device), group=group, dtype=F32).cpu()]
        y, size = product64(s["x"], s["w"][1], s["ws"][1].float().clamp(-1, 1), group)
        for out in got:
            assert torch.equal(out[:, ~other], want[~other].expand(tokens, -1))
            check(out[:, other], *(t[:, other] for t in bounded(y, size, parts(k, group), None, None, F32)))


@pytest.mark.parametrize("tokens", [1, 8, 9, 40, 129, 300, 1000])
def test_vanishing_activation_scales(loom, device, tokens):  # noqa: F811
    """Scales of rows that are all but zero lie below the smallest normal f32: they are used as they are.  Sums and results
    here are whole multiples of powers of two, so they are exact in f32."""
    rows, k, group = 1100, 320, 128
    g = torch.Generator().manual_seed(tokens)
    wq = torch.randint(-8, 8, (2, rows, k), generator=g, dtype=torch.int8)
    xq = torch.randint(-20, 21, (tokens, k), generator=g, dtype=torch.int8)
    ws = torch.full((2, rows, 3), 2.0 ** 100)
    step = 2.0 ** -149
    xs = (torch.randint(1, 8, (tokens,), generator=g).double() * step).float()
    w, x = loom.pack_int4(wq.to(device)), loom.pack_int8(xq.to(device))
    offsets = offsets_of([0, tokens]).to(device)
    want = (xq.double() @ wq[1].double().t()) * 2.0 ** 100 * xs.double()[:, None]
    got = [loom.i4_matmul(w[1], ws[1].to(device), x, xs.to(device), group=group, dtype=F32),
           loom.i4_expert_matmul(w, ws.to(device), x, xs.to(device), offsets, group=group, dtype=F32),
           loom.i4_expert_gated_projection(w, ws.to(device), w, ws.to(device), x, xs.to(device), offsets, act="relu", group=group,
                                           dtype=F32)]
    assert bool((xs > 0).all()) and torch.equal(got[0].cpu().double(), want) and torch.equal(got[1].cpu().double(), want)
    both = want.clamp(min=0) * want  # about 2^-60: one rounding
    assert bool(((got[2].cpu().double() - both).abs() <= 2.0 ** -24 * both.abs()).all())


@pytest.mark.parametrize("tokens", [1, 8, 9, 40, 129, 300, 1000])
def test_large_sums(loom, device, tokens):  # noqa: F811
    """Sums of just less than 2^124, before an activation's scale brings them back, are exact too."""
    rows, k, group = 1100, 320, 128
    g = torch.Generator().manual_seed(tokens)
    wq = torch.randint(-8, 8, (rows, k), generator=g, dtype=torch.int8)
    xq = torch.randint(-20, 21, (tokens, k), generator=g, dtype=torch.int8)
    ws, xs = torch.full((rows, 3), 2.0 ** 108), torch.full((tokens,), 2.0 ** -90)
    assert 8 * 20 * k < 2 ** 16
    want = (xq.double() @ wq.double().t()) * 2.0 ** 18
    got = loom.i4_matmul(loom.pack_int4(wq.to(device)), ws.to(device), loom.pack_int8(xq.to(device)), xs.to(device), group=group,
                         dtype=F32)
    assert torch.equal(got.cpu().double(), want)


# ------------------------------------------------------------------ offsets that overlap

@pytest.mark.parametrize("pairs,offsets", [(200, [0, 150, 0, 200]), (200, [0, 200, 0, 200, 0, 200, 190]), (7, [0, 7, 2, 6, 0, 7]),
                                           (300, [200, 300, 0, 50, 20, 300]),
                                           (300, [100, 200, 0, 50, 20, 40])])
def test_overlapping_offsets(loom, device, pairs, offsets):  # noqa: F811
    """Where ranges overlap, every element of a claimed row is as it was or one claimant's; no other row is written."""
    experts, rows, k, group = len(offsets) - 1, 200, 64, 32
    s = operands(experts, rows, k, pairs, group, F32, 3)
    d = {n: t.to(device) for n, t in s.items()}
    out = torch.full((pairs, rows), 7.0, device=device)
    loom.i4_expert_matmul(loom.pack_int4(d["w"]), d["ws"], loom.pack_int8(d["x"]), d["xs"],
                          torch.tensor(offsets, dtype=torch.int32, device=device), group=group, out=out)
    out = out.cpu().double()
    fits = out == 7.0
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            y, size = product64(s["x"][a:b], s["w"][e], s["ws"][e], group)
            v, tol = bounded(y, size, parts(k, group), s["xs"][a:b], None, F32)
            fits[a:b] |= (out[a:b] - v).abs() <= tol
    assert bool(fits.all())


def test_scales_of_other_groups(loom, device):  # noqa: F811
    """Scales made for another group length are refused; a longer flat buffer is read from its start."""
    s = operands(2, 40, 256, 5, 32, F32, 1)
    d = {n: t.to(device) for n, t in s.items()}
    w, x, off = loom.pack_int4(d["w"]), loom.pack_int8(d["x"]), offsets_of([2, 3]).to(device)
    for group in (64, 128, 256):
        with pytest.raises(ValueError, match="scales a channel"):
            loom.i4_matmul(w[0], d["ws"][0], x, group=group)
        with pytest.raises(ValueError, match="scales a channel"):
            loom.i4_expert_matmul(w, d["ws"], x, None, off, group=group)
        with pytest.raises(ValueError, match="scales a channel"):
            loom.i4_expert_gated_projection(w, d["ws"], w, d["ws"], x, None, off, group=group)
    want = loom.i4_matmul(w[0], d["ws"][0], x, group=32)
    assert torch.equal(loom.i4_matmul(w[0], d["ws"].flatten(), x, group=32), want)
