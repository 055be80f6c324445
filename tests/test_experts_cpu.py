"""The argument contract of the router, its gradient, route grouping and the 4-bit products, on the host: statuses of
random calls against the rules of include/loom.h, launch geometry, packing, and the refusals that need no GPU."""
import ctypes

import pytest
import torch
from hypothesis import given, strategies as st

from tests.test_abi_contract import (I31, I64, NULL, OK, PTRS, RANGE, SETTINGS, SHAPE, _grid_refused, _mis, _no_gpu, _p,
                                     _status, sizes)

no_gpu = pytest.mark.skipif(not _no_gpu(), reason="a passing call would launch on placeholder pointers")
TYPES = st.sampled_from([-1, 0, 1, 2, 3])
SCORES = st.sampled_from([-1, 0, 1, 2])
GROUPS = st.sampled_from([-1, 0, 16, 31, 32, 48, 64, 128, 2 ** 17, 2 ** 17 + 1, 2 ** 18])
SMALL = dict(tokens=sizes(I31, 2 ** 26), stride=sizes(I31, 2 ** 40))


@pytest.fixture(scope="module")
def loom():
    import int8_dequant_dot_amd as m
    return m


@pytest.fixture(scope="module")
def lib(loom):
    return loom.library()


def _size(kind):
    return 4 if kind == 0 else 2


def _route_rules(tokens, experts, groups, top_k, kind, score, stride, export):
    fine = (0 <= tokens <= I31 and 0 <= kind <= 2 and 0 <= score <= 1 and 1 <= experts <= 1024 and 1 <= groups <= 64
            and 1 <= top_k <= 64)
    return [(RANGE, not fine), (SHAPE, stride < experts or top_k > experts), (RANGE, tokens > 0 and 4 * tokens * stride > I64),
            (RANGE, fine and _grid_refused(export, [tokens, experts, groups, top_k]))]


@no_gpu
@SETTINGS
@given(l=PTRS, bias=PTRS, ids=PTRS, w=PTRS, kind=TYPES, score=SCORES, experts=sizes(1024), groups=sizes(64), kept=sizes(64),
       top=st.sampled_from([0, 1, 2, 3]), top_k=sizes(64), **SMALL)
def test_route_experts_contract(lib, l, bias, ids, w, kind, score, experts, groups, kept, top, top_k, tokens, stride):
    divides = groups > 0 and experts % groups == 0
    expect = _status([(RANGE, top not in (1, 2))] + _route_rules(tokens, experts, groups, top_k, kind, score, stride, "route_experts")
                     + [(RANGE, not 1 <= kept <= groups), (SHAPE, not divides or top_k > kept * (experts // max(groups, 1)))],
                     tokens == 0, None in (l, ids, w), _mis(l, _size(kind)) or any(_mis(p, 4) for p in (bias, ids, w)))
    assert lib.loom_route_experts(_p(l), kind, tokens, experts, stride, score, _p(bias), groups, kept, top, top_k, 1, 1.0,
                                  _p(ids), _p(w), None) == expect


@no_gpu
@SETTINGS
@given(l=PTRS, ids=PTRS, d=PTRS, dl=PTRS, kind=TYPES, score=SCORES, experts=sizes(1024), top_k=sizes(64),
       d_stride=sizes(I31, 2 ** 40), **SMALL)
def test_route_experts_backward_contract(lib, l, ids, d, dl, kind, score, experts, top_k, d_stride, tokens, stride):
    expect = _status(_route_rules(tokens, experts, 1, top_k, kind, score, stride, "route_experts_backward")
                     + [(SHAPE, d_stride < experts), (RANGE, tokens > 0 and 4 * tokens * d_stride > I64)],
                     tokens == 0, None in (l, ids, d, dl),
                     _mis(l, _size(kind)) or _mis(dl, _size(kind)) or any(_mis(p, 4) for p in (ids, d)))
    assert lib.loom_route_experts_backward(_p(l), kind, tokens, experts, stride, score, top_k, 0, 1.0, _p(ids), _p(d),
                                           _p(dl), d_stride, None) == expect


@no_gpu
@SETTINGS
@given(ids=PTRS, slots=PTRS, rows=PTRS, off=PTRS, space=PTRS, tokens=sizes(I31, 2 ** 26), routes=sizes(2 ** 20, 64),
       experts=sizes(1024), short=st.booleans())
def test_group_routes_contract(lib, ids, slots, rows, off, space, tokens, routes, experts, short):
    fine = 0 <= tokens <= I31 and 0 <= routes <= 2 ** 20 and tokens * routes <= I31 and 1 <= experts <= 1024
    need = ctypes.c_int64(-1)
    said = lib.loom_group_routes_workspace(tokens, routes, experts, ctypes.byref(need))
    assert said == (OK if fine else RANGE) and (need.value >= 0 or said != OK)
    pairs = tokens * routes
    expect = _status([(RANGE, not fine), (RANGE, short)], False,
                     off is None or (pairs > 0 and None in (ids, slots, rows)) or (need.value > 0 and space is None),
                     any(_mis(p, 4) for p in (ids, slots, rows, off, space)))
    assert lib.loom_group_routes(_p(ids), tokens, routes, experts, _p(slots), _p(rows), _p(off), _p(space),
                                 need.value - 1 if short else max(need.value, 0), None) == expect


def _product_rules(rows, k, tokens, group, kind, scales, stride, export, experts=None):
    fine = (0 <= k <= 131040 and 0 <= rows <= I31 and 0 <= tokens <= I31 and 0 <= kind <= 2 and 0 <= scales <= 2
            and 32 <= group <= 2 ** 17 and (experts is None or 1 <= experts <= 1024))
    load = [rows, k, tokens, group] + ([] if experts is None else [experts])
    return [(RANGE, not fine), (SHAPE, k % 32 != 0 or group & (group - 1) != 0 or stride < rows),
            (RANGE, tokens > 0 and 4 * tokens * stride > I64), (RANGE, fine and _grid_refused(export, load))]


SIZES = dict(kind=TYPES, scales=TYPES, group=GROUPS, rows=sizes(I31, 2 ** 26), k=st.one_of(sizes(131040, 131072), st.sampled_from([32, 64, 4096])),
             tokens=sizes(I31, 2 ** 26), stride=sizes(I31, 2 ** 40))


@no_gpu
@SETTINGS
@given(w=PTRS, ws=PTRS, x=PTRS, xs=PTRS, bias=PTRS, out=PTRS, **SIZES)
def test_i4_matmul_contract(lib, w, ws, x, xs, bias, out, kind, scales, group, rows, k, tokens, stride):
    expect = _status(_product_rules(rows, k, tokens, group, kind, scales, stride, "i4_matmul"), rows == 0 or tokens == 0,
                     out is None or (k > 0 and None in (w, ws, x)),
                     _mis(w, 16) or _mis(x, 16) or _mis(ws, _size(scales)) or _mis(xs, 4) or _mis(bias, 4) or _mis(out, _size(kind)))
    assert lib.loom_i4_matmul(_p(w), _p(ws), scales, group, _p(x), _p(xs), _p(bias), rows, k, tokens, _p(out), kind, stride,
                              None) == expect


@no_gpu
@SETTINGS
@given(w=PTRS, ws=PTRS, u=PTRS, us=PTRS, x=PTRS, xs=PTRS, index=PTRS, off=PTRS, bias=PTRS, out=PTRS, experts=sizes(1024),
       x_rows=sizes(I31), act=st.sampled_from([-1, 0, 3, 4]), **SIZES)
def test_experts_products_contract(lib, w, ws, u, us, x, xs, index, off, bias, out, experts, x_rows, act, kind, scales, group,
                                   rows, k, tokens, stride):
    def rules(name):
        return (_product_rules(rows, k, tokens, group, kind, scales, stride, name, experts)
                + [(RANGE, not 0 <= x_rows <= I31), (SHAPE, tokens > 0 and x_rows < (tokens if index is None else 1))])
    odd = (_mis(w, 16) or _mis(x, 16) or _mis(ws, _size(scales)) or any(_mis(p, 4) for p in (xs, index, off))
           or _mis(out, _size(kind)))
    nothing = rows == 0 or tokens == 0
    missing = out is None or off is None or (k > 0 and None in (w, ws, x))
    assert lib.loom_i4_expert_matmul(_p(w), _p(ws), scales, group, _p(x), _p(xs), x_rows, _p(index), _p(off), _p(bias), experts,
                                     rows, k, tokens, _p(out), kind, stride, None) == _status(
        rules("i4_expert_matmul"), nothing, missing, odd or _mis(bias, 4))
    assert lib.loom_i4_expert_gated_projection(_p(w), _p(ws), _p(u), _p(us), scales, group, _p(x), _p(xs), x_rows, _p(index),
                                               _p(off), experts, rows, k, tokens, act, _p(out), kind, stride, None) == _status(
        [(RANGE, not 0 <= act <= 3)] + rules("i4_expert_gated_projection"), nothing,
        missing or (k > 0 and None in (u, us)), odd or _mis(u, 16) or _mis(us, _size(scales)))


def test_workspace_needs_its_result(lib):
    assert lib.loom_group_routes_workspace(8, 8, 8, None) == NULL


@pytest.mark.parametrize("name,load", [("route_experts", [1, 64, 8, 8]), ("route_experts_backward", [1, 64, 1, 8]),
                                       ("group_routes", [8, 64]), ("i4_matmul", [64, 128, 1, 32]),
                                       ("i4_expert_matmul", [64, 128, 1, 32, 8]),
                                       ("i4_expert_gated_projection", [64, 128, 1, 32, 8])])
def test_launch_geometry(loom, name, load):
    token = loom.launch_config_lookup(name)
    for bad in (load[:-1], load + [1]):
        with pytest.raises(loom.LoomError) as e:
            loom.launch_config_invoke(token, bad)
        assert e.value.status == loom.ERR_TOKEN
    for i in range(len(load)):
        with pytest.raises(loom.LoomError):
            loom.launch_config_invoke(token, load[:i] + [-1] + load[i + 1:])

    def fits(work, some=True):
        c = loom.launch_config_invoke(token, work)
        wg = c["workgroups"]
        assert wg[0] * wg[1] * wg[2] > 0 or not some
        assert c["workgroup_size"][0] % 64 == 0 and c["workgroup_size"][0] <= 1024
        assert c["workgroup_storage_bytes"] <= 160 * 1024
    counts = (1, 7, 16, 17, 33, 64, 129, 1023, 1024, 100000, 2 ** 24)
    if name.startswith("route"):
        for tokens in counts + (I31,):
            for experts in (1, 64, 255, 256, 257, 1024):
                for groups, top_k in ((1, 1), (64, 64), (8, 16), (8, 17)):
                    fits([tokens, experts, groups, top_k])
        fits([0, 64, 1, 8], False)
    elif name == "group_routes":
        for pairs in (0,) + counts + (I31,):
            for experts in (1, 256, 1024):
                fits([pairs, experts])
    else:
        for rows in (1, 15, 16, 17, 4099, 28672):
            for k in (0, 32, 512, 8192, 131040):
                for tokens in counts[:-1]:
                    for group in (32, 64, 128, 2 ** 17):
                        for experts in (1, 8, 1024):
                            fits([rows, k, tokens, group] + ([experts] if name != "i4_matmul" else []))


@pytest.mark.parametrize("name", ["i4_matmul", "i4_expert_matmul", "i4_expert_gated_projection"])
def test_nothing_to_do_has_no_grid(loom, name):
    token = loom.launch_config_lookup(name)
    for rows, k, tokens in ((64, 128, 0), (0, 128, 5), (0, 0, 0)):
        for group in (32, 128):
            work = [rows, k, tokens, group] + ([] if name == "i4_matmul" else [8])
            assert loom.launch_config_invoke(token, work)["workgroups"][0] == 0


def test_pack_int4(loom):
    g = torch.Generator().manual_seed(0)
    for shape in ((1, 32), (3, 96), (2, 5, 64), (4, 0), (0, 64)):
        q = torch.randint(-8, 8, shape, generator=g, dtype=torch.int8)
        w = loom.pack_int4(q)
        assert w.dtype == torch.int32 and tuple(w.shape) == (*shape[:-1], shape[-1] // 8)
        if not q.numel():
            continue
        b = w.contiguous().view(torch.uint8).view(*shape[:-1], shape[-1] // 32, 16).to(torch.int16)
        back = torch.empty(*shape[:-1], shape[-1] // 32, 32, dtype=torch.int16)
        for i in range(16):  # the documented layout, byte by byte
            back[..., i], back[..., 16 + i] = b[..., i] & 15, b[..., i] >> 4
        back = torch.where(back > 7, back - 16, back).view(shape)
        assert torch.equal(back, q.to(torch.int16))
    strided = torch.randint(-8, 8, (64, 4), generator=g, dtype=torch.int8).t()
    assert torch.equal(loom.pack_int4(strided), loom.pack_int4(strided.contiguous()))
    for bad in (torch.zeros(2, 40, dtype=torch.int8), torch.zeros(2, 32, dtype=torch.int16)):
        with pytest.raises(ValueError):
            loom.pack_int4(bad)


def test_cpu_tensors_and_names_are_refused(loom):
    l = torch.zeros(2, 8)
    ids = torch.zeros(2, 2, dtype=torch.int32)
    w = torch.zeros(4, 4, dtype=torch.int32)
    for call in (lambda: loom.route_experts(l, 2), lambda: loom.route_experts_backward(l, ids, l[:, :2]),
                 lambda: loom.group_routes(ids, 8), lambda: loom.i4_matmul(w, l, w), lambda: loom.i4_expert_matmul(w, l, w, l, ids),
                 lambda: loom.i4_expert_gated_projection(w, l, w, l, w, l, ids)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(loom.LoomError):
        loom.group_routes_workspace(8, 8, 0)
