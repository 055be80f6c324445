"""The int8 feed-forward operators' argument contract, on the host: statuses of random calls against the rules of
include/loom.h, launch geometry, and the binding's refusals that need no GPU."""
import ctypes

import pytest
import torch
from hypothesis import given, strategies as st

from tests.test_abi_contract import (I31, I64, NULL, OK, PTRS, RANGE, SETTINGS, SHAPE, _grid_refused, _mis, _no_gpu, _p,
                                     _status, sizes)

no_gpu = pytest.mark.skipif(not _no_gpu(), reason="a passing call would launch on placeholder pointers")
TYPES = st.sampled_from([-1, 0, 1, 2, 3])
ACTS = st.sampled_from([-1, 0, 1, 2, 3, 4])


@pytest.fixture(scope="module")
def loom():
    import int8_dequant_dot_amd as m
    return m


@pytest.fixture(scope="module")
def lib(loom):
    return loom.library()


def _size(kind):
    return 4 if kind == 0 else 2


@no_gpu
@SETTINGS
@given(x=PTRS, q=PTRS, scale=PTRS, kind=TYPES, rows=sizes(I31, 2**30), cols=sizes(I31, 2**30), stride=sizes(I31, 2**40))
def test_quantize_rows_contract(lib, x, q, scale, kind, rows, cols, stride):
    expect = _status([(RANGE, not (0 <= rows <= I31 and 0 <= cols <= I31 and 0 <= kind <= 2)),
                      (SHAPE, cols % 4 != 0 or stride < cols), (RANGE, rows > 0 and 4 * rows * stride > I64),
                      (RANGE, rows >= 0 and cols >= 0 and _grid_refused("quantize_rows", [rows, cols]))],
                     rows == 0, scale is None or (cols > 0 and (x is None or q is None)),
                     _mis(x, _size(kind)) or _mis(q, 4) or _mis(scale, 4))
    assert lib.loom_quantize_rows(_p(x), kind, rows, cols, stride, _p(q), _p(scale), None) == expect


def _product_rules(rows, k, tokens, kind, stride, export, act=0):
    fine = (0 <= k <= 131068 and 0 <= rows <= I31 and 0 <= tokens <= I31 and 0 <= kind <= 2 and 0 <= act <= 3)
    return [(RANGE, not fine), (SHAPE, k % 4 != 0 or stride < rows), (RANGE, tokens > 0 and 4 * tokens * stride > I64),
            (RANGE, fine and _grid_refused(export, [rows, k, tokens]))]


SIZES = dict(kind=TYPES, rows=sizes(I31, 2**26), k=sizes(131068), tokens=sizes(I31, 2**26), stride=sizes(I31, 2**40))


@no_gpu
@SETTINGS
@given(w=PTRS, ws=PTRS, x=PTRS, xs=PTRS, bias=PTRS, out=PTRS, **SIZES)
def test_i8_matmul_contract(lib, w, ws, x, xs, bias, out, kind, rows, k, tokens, stride):
    expect = _status(_product_rules(rows, k, tokens, kind, stride, "i8_matmul"), rows == 0 or tokens == 0,
                     ws is None or out is None or (k > 0 and (w is None or x is None)),
                     any(_mis(p, 4) for p in (w, ws, x, xs, bias)) or _mis(out, _size(kind)))
    assert lib.loom_i8_matmul(_p(w), _p(ws), _p(x), _p(xs), _p(bias), rows, k, tokens, _p(out), kind, stride,
                              None) == expect


@no_gpu
@SETTINGS
@given(w=PTRS, ws=PTRS, u=PTRS, us=PTRS, x=PTRS, xs=PTRS, out=PTRS, act=ACTS, **SIZES)
def test_i8_gated_projection_contract(lib, w, ws, u, us, x, xs, out, act, kind, rows, k, tokens, stride):
    expect = _status(_product_rules(rows, k, tokens, kind, stride, "i8_gated_projection", act),
                     rows == 0 or tokens == 0,
                     ws is None or us is None or out is None or (k > 0 and (w is None or u is None or x is None)),
                     any(_mis(p, 4) for p in (w, ws, u, us, x, xs)) or _mis(out, _size(kind)))
    assert lib.loom_i8_gated_projection(_p(w), _p(ws), _p(u), _p(us), _p(x), _p(xs), rows, k, tokens, act, _p(out),
                                        kind, stride, None) == expect


@no_gpu
@SETTINGS
@given(w=PTRS, ws=PTRS, u=PTRS, us=PTRS, x=PTRS, xs=PTRS, d=PTRS, dx=PTRS, dg=PTRS, du=PTRS, space=PTRS, act=ACTS,
       short=st.booleans(), **SIZES)
def test_i8_gated_projection_backward_contract(lib, w, ws, u, us, x, xs, d, dx, dg, du, space, act, short, kind, rows,
                                               k, tokens, stride):
    name = "i8_gated_projection_backward"
    need = ctypes.c_int64(-1)
    said = lib.loom_i8_gated_projection_backward_workspace(rows, k, tokens, kind, ctypes.byref(need))
    assert said == _status(_product_rules(rows, k, tokens, kind, rows, name), True, False, False)
    assert need.value >= 0 or said != OK
    given_bytes = need.value - 1 if short else max(need.value, 0)
    live = rows > 0 and tokens > 0
    expect = _status(_product_rules(rows, k, tokens, kind, stride, name, act) + [(RANGE, short)],
                     (dx is None or tokens == 0 or k == 0) and ((dg is None and du is None) or rows == 0),
                     live and (None in (ws, us, d, space) or (k > 0 and None in (w, u, x))),
                     any(_mis(p, 4) for p in (w, ws, u, us, x, xs, dg, du)) or _mis(d, _size(kind))
                     or _mis(dx, _size(kind)) or _mis(space, 16))
    assert lib.loom_i8_gated_projection_backward(_p(w), _p(ws), _p(u), _p(us), _p(x), _p(xs), rows, k, tokens, act,
                                                 _p(d), kind, stride, _p(dx), _p(dg), _p(du), _p(space), given_bytes,
                                                 None) == expect


def test_workspace_needs_its_result(lib):
    assert lib.loom_i8_gated_projection_backward_workspace(8, 8, 8, 0, None) == NULL


@pytest.mark.parametrize("name", ["quantize_rows", "i8_matmul", "i8_gated_projection", "i8_gated_projection_backward"])
def test_launch_geometry(loom, name):
    token = loom.launch_config_lookup(name)
    arity = 2 if name == "quantize_rows" else 3
    for bad in ([1] * (arity - 1), [1] * (arity + 1)):
        with pytest.raises(loom.LoomError) as e:
            loom.launch_config_invoke(token, bad)
        assert e.value.status == loom.ERR_TOKEN
    with pytest.raises(loom.LoomError):
        loom.launch_config_invoke(token, [-1] + [4] * (arity - 1))
    assert loom.launch_config_invoke(token, [0] + [64] * (arity - 1))["workgroups"][0] == 0
    # any size the entry points take without a refusal has a grid and LDS that fit the hardware
    for rows in (1, 15, 16, 17, 4099, 28672):
        for k in (0, 4, 60, 64, 1024, 8192, 131068):
            for tokens in (1, 2, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 4096, 100000):
                c = loom.launch_config_invoke(token, [rows, k] if arity == 2 else [rows, k, tokens])
                wg = c["workgroups"]
                assert wg[0] * wg[1] * wg[2] > 0 and c["workgroup_size"][0] % 64 == 0
                assert c["workgroup_size"][0] <= 1024 and c["workgroup_storage_bytes"] <= 160 * 1024


def test_cpu_tensors_and_names_are_refused(loom):
    w = torch.zeros(4, 4, dtype=torch.int32)
    s = torch.zeros(4)
    with pytest.raises(TypeError):
        loom.quantize_rows(torch.zeros(2, 8))
    with pytest.raises(TypeError):
        loom.i8_matmul(w, s, w, s)
    with pytest.raises(TypeError):
        loom.i8_gated_projection(w, s, w, s, w, s)
    with pytest.raises(TypeError):
        loom.i8_gated_projection_backward(w, s, w, s, w, s, torch.zeros(4, 4))
    with pytest.raises(TypeError):
        loom.i8_gated_projection_backward_workspace(8, 8, 8, torch.float64)
    with pytest.raises(loom.LoomError):
        loom.i8_gated_projection_backward_workspace(8, 6, 8)
