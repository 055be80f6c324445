"""Python binding of the MI355X streaming-reduction library (``libloom.so``).

Argument marshalling only: every step of the computation runs in the gfx950 HIP
kernels behind the C ABI declared in ``include/loom.h``.  PyTorch supplies device
memory and the stream (``torch.cuda.current_stream()``).  There is no CPU
fallback: if the HIP library is missing, importing this package raises.

Functions carry the C entry points' names without the ``loom_`` prefix.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # load torch's HIP runtime first so libloom.so binds to the same instance

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libloom.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_lib.loom_status_string.restype = ctypes.c_char_p
_lib.loom_status_string.argtypes = [ctypes.c_int]
_lib.loom_version.restype = ctypes.c_int
_lib.loom_version.argtypes = []
_lib.loom_launch_config_lookup.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_uint32)]
_lib.loom_launch_config_invoke.argtypes = [ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64), ctypes.c_size_t, _p]
_lib.loom_copy_f32.argtypes = [_p, _p, _i64, _p]
_lib.loom_row_sum_tiles.argtypes = [_p, _i64, _i64, _p, _p, _p, _p, _p]
_lib.loom_row_sums.argtypes = [_p, _i64, _i64, _i64, _p, _p]
_lib.loom_segment_sums.argtypes = [_p, _i64, _p, _i64, _i64, _p, _p, _p]
_lib.loom_segment_sums_noalloc.argtypes = [_p, _i64, _p, _i64, _i64, _p, _p, _p]
_lib.loom_i8_dequant_dot.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p]
_lib.loom_packed_dot.argtypes = [_p, _p, _p, _i64, _p, _i64, _i64, _i64, _p, _p]
_lib.loom_sum_guarded_rows.argtypes = [_p, _i64, _i64, _i64, _i64, _p, _p]
_lib.loom_routed_combine.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i64, _p, _p]
_lib.loom_quantize_rows.argtypes = [_p, ctypes.c_int, _i64, _i64, _i64, _p, _p, _p]
_lib.loom_i8_matmul.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_int, _i64, _p]
_lib.loom_i8_gated_projection.argtypes = [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, ctypes.c_int, _p, ctypes.c_int,
                                          _i64, _p]
_lib.loom_i8_gated_projection_backward_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int, _p]
_lib.loom_i8_gated_projection_backward.argtypes = [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, ctypes.c_int, _p,
                                                   ctypes.c_int, _i64, _p, _p, _p, _p, _i64, _p]
_int, _float = ctypes.c_int, ctypes.c_float
_lib.loom_route_experts.argtypes = [_p, _int, _i64, _i64, _i64, _int, _p, _i64, _i64, _i64, _i64, _int, _float, _p, _p,
                                    _p]
_lib.loom_route_experts_backward.argtypes = [_p, _int, _i64, _i64, _i64, _int, _i64, _int, _float, _p, _p, _p, _i64, _p]
_lib.loom_group_routes_workspace.argtypes = [_i64, _i64, _i64, _p]
_lib.loom_group_routes.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _p]
_lib.loom_i4_matmul.argtypes = [_p, _p, _int, _i64, _p, _p, _p, _i64, _i64, _i64, _p, _int, _i64, _p]
_lib.loom_i4_expert_matmul.argtypes = [_p, _p, _int, _i64, _p, _p, _i64, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _int,
                                       _i64, _p]
_lib.loom_i4_expert_gated_projection.argtypes = [_p, _p, _p, _p, _int, _i64, _p, _p, _i64, _p, _p, _i64, _i64, _i64,
                                                 _i64, _int, _p, _int, _i64, _p]
for _name in ("loom_launch_config_lookup", "loom_launch_config_invoke", "loom_copy_f32", "loom_row_sum_tiles",
              "loom_row_sums", "loom_segment_sums", "loom_segment_sums_noalloc", "loom_i8_dequant_dot",
              "loom_packed_dot",
              "loom_sum_guarded_rows", "loom_routed_combine", "loom_quantize_rows", "loom_i8_matmul",
              "loom_i8_gated_projection", "loom_i8_gated_projection_backward_workspace",
              "loom_i8_gated_projection_backward", "loom_route_experts", "loom_route_experts_backward",
              "loom_group_routes_workspace", "loom_group_routes", "loom_i4_matmul", "loom_i4_expert_matmul",
              "loom_i4_expert_gated_projection"):
    getattr(_lib, _name).restype = ctypes.c_int

# status codes (include/loom.h)
OK, ERR_NULL, ERR_RANGE, ERR_ALIGN, ERR_SHAPE, ERR_UNKNOWN_EXPORT, ERR_TOKEN, ERR_DEVICE = 0, -1, -2, -3, -4, -5, -6, -7

EXPORTS = ("copy_f32", "row_sum_tiles", "row_sums", "segment_sums", "i8_dequant_dot", "packed_dot",
           "sum_guarded_rows", "routed_combine", "quantize_rows", "i8_matmul", "i8_gated_projection",
           "i8_gated_projection_backward", "route_experts", "route_experts_backward", "group_routes", "i4_matmul",
           "i4_expert_matmul", "i4_expert_gated_projection")

# loom_type and loom_activation (include/loom.h)
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
SCORES = {"softmax": 0, "sigmoid": 1}  # loom_score


class LoomError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class LaunchConfig(ctypes.Structure):
    _fields_ = [("workgroups", ctypes.c_uint32 * 3), ("workgroup_size", ctypes.c_uint32 * 3),
                ("cluster_size", ctypes.c_uint32 * 3), ("subgroup_size", ctypes.c_uint32),
                ("workgroup_storage_bytes", ctypes.c_uint32)]

    def as_dict(self):
        return {"workgroups": tuple(self.workgroups), "workgroup_size": tuple(self.workgroup_size),
                "cluster_size": tuple(self.cluster_size), "subgroup_size": self.subgroup_size,
                "workgroup_storage_bytes": self.workgroup_storage_bytes}


def library():
    """The loaded ctypes library (for tests that call the C ABI directly)."""
    return _lib


def status_string(status: int) -> str:
    return _lib.loom_status_string(status).decode()


def version() -> int:
    return _lib.loom_version()


def _check(status: int, where: str):
    if status != OK:
        raise LoomError(status, where)


def launch_config_lookup(export_name: str) -> int:
    tok = ctypes.c_uint32()
    _check(_lib.loom_launch_config_lookup(export_name.encode(), ctypes.byref(tok)), "launch_config_lookup")
    return tok.value


def launch_config_invoke(token: int, workload) -> dict:
    vals = [int(v) & ((1 << 64) - 1) for v in workload]
    arr = (ctypes.c_uint64 * max(1, len(vals)))(*vals)
    cfg = LaunchConfig()
    _check(_lib.loom_launch_config_invoke(token, arr, len(vals), ctypes.byref(cfg)), "launch_config_invoke")
    return cfg.as_dict()


# ------------------------------------------------------------------ tensor helpers

# the current stream's handle without a Stream object around it (1.1 us a call), where this torch has that call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _target(t: torch.Tensor, name: str):
    """The current HIP device index and its current stream: the C ABI launches
    there, so every tensor must live on that device.  ``t`` (the call's first
    tensor) is checked first, so a CPU tensor is refused before any HIP call."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    device = torch.cuda.current_device()
    return device, _raw_stream(device)


def _dev(t: torch.Tensor, dtype, name: str, device: int) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _buffer(t: torch.Tensor | None, dtype, numel: int, name: str, device: int, optional: bool = False):
    """A caller-supplied input or output buffer: a contiguous device tensor of `dtype` holding at
    least `numel` elements (the kernels read or write that many from its start)."""
    if t is None:
        if not optional:
            raise ValueError(f"{name} is required")
        return None
    _dev(t, dtype, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, {numel} are needed")
    return t


def copy_f32(inp: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """out[i] = inp[i] for i < inp.numel(); elements of ``out`` beyond that are untouched."""
    device, stream = _target(inp, "inp")
    _dev(inp, torch.float32, "inp", device)
    _require(inp.is_contiguous(), "inp must be contiguous")
    if out is None:
        out = torch.empty_like(inp)
    _buffer(out, torch.float32, inp.numel(), "out", device)
    _check(_lib.loom_copy_f32(_ptr(inp), _ptr(out), inp.numel(), stream), "copy_f32")
    return out


def row_sum_tiles(values: torch.Tensor, count: int, initial: torch.Tensor | None = None):
    """values [rows_alloc][32] f32 -> (sums[32] f32, final_row int32[1], tail_count int32[1])."""
    device, stream = _target(values, "values")
    _dev(values, torch.float32, "values", device)
    _require(values.dim() == 2 and values.shape[1] == 32 and values.is_contiguous(),
             "values must be a contiguous [rows][32] tensor")
    _buffer(initial, torch.float32, 32, "initial", device, optional=True)
    sums = torch.empty(32, dtype=torch.float32, device=values.device)
    fr = torch.empty(1, dtype=torch.int32, device=values.device)
    tc = torch.empty(1, dtype=torch.int32, device=values.device)
    _check(_lib.loom_row_sum_tiles(_ptr(values), values.shape[0], count, _ptr(initial), _ptr(sums), _ptr(fr),
                                   _ptr(tc), stream), "row_sum_tiles")
    return sums, fr, tc


def row_sums(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """x [rows][cols] f32 with unit column stride (any row stride) -> out [rows]."""
    device, stream = _target(x, "x")
    _dev(x, torch.float32, "x", device)
    _require(x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] <= 1), "x must be [rows][cols] with unit column stride")
    rows, cols = x.shape
    stride = x.stride(0) if rows > 1 else max(cols, 1)
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=x.device)
    _buffer(out, torch.float32, rows, "out", device)
    _check(_lib.loom_row_sums(_ptr(x), rows, cols, stride, _ptr(out), stream), "row_sums")
    return out


def segment_sums(x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                 tail_counts: torch.Tensor | None = None, want_tails: bool = True, noalloc: bool = False):
    """x [total_rows][cols] f32, offsets int64 [S+1] (CSR) -> (out [S][cols], tail_counts int32 [S]).

    noalloc=True calls loom_segment_sums_noalloc (no device allocation inside
    the call; calls that overlap on one GPU must be ordered by the caller)."""
    device, stream = _target(x, "x")
    _dev(x, torch.float32, "x", device)
    _dev(offsets, torch.int64, "offsets", device)
    _require(x.dim() == 2 and x.is_contiguous(), "x must be a contiguous [total_rows][cols] tensor")
    _require(offsets.dim() == 1 and offsets.is_contiguous() and offsets.numel() >= 1,
             "offsets must be a contiguous [segments + 1] tensor")
    S = offsets.numel() - 1
    cols = x.shape[1]
    if out is None:
        out = torch.empty(S, cols, dtype=torch.float32, device=x.device)
    _buffer(out, torch.float32, S * cols, "out", device)
    if tail_counts is None and want_tails:
        tail_counts = torch.empty(S, dtype=torch.int32, device=x.device)
    _buffer(tail_counts, torch.int32, S, "tail_counts", device, optional=True)
    fn = _lib.loom_segment_sums_noalloc if noalloc else _lib.loom_segment_sums
    _check(fn(_ptr(x), x.shape[0], _ptr(offsets), S, cols, _ptr(out), _ptr(tail_counts), stream),
           "segment_sums_noalloc" if noalloc else "segment_sums")
    return out, tail_counts


def i8_dequant_dot(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, acc: torch.Tensor | None = None, want_acc: bool = False):
    """w int32 [rows][k/4] (packed int8), x int32 [batch][k/4] or [k/4] -> out f32 [rows][batch] (and acc)."""
    device, stream = _target(w, "w")
    _dev(w, torch.int32, "w", device)
    _dev(x, torch.int32, "x", device)
    if x.dim() == 1:
        x = x.view(1, -1)
    _require(w.dim() == 2 and w.is_contiguous(), "w must be a contiguous [rows][k/4] tensor")
    _require(x.dim() == 2 and x.is_contiguous() and x.shape[1] == w.shape[1],
             "x must be a contiguous [batch][k/4] tensor with the same k as w")
    rows, kw = w.shape
    batch = x.shape[0]
    _buffer(w_scale, torch.float32, rows, "w_scale", device)
    _buffer(x_scale, torch.float32, batch, "x_scale", device, optional=True)
    if out is None:
        out = torch.empty(rows, batch, dtype=torch.float32, device=w.device)
    _buffer(out, torch.float32, rows * batch, "out", device)
    if acc is None and want_acc:
        acc = torch.empty(rows, batch, dtype=torch.int32, device=w.device)
    _buffer(acc, torch.int32, rows * batch, "acc", device, optional=True)
    _check(_lib.loom_i8_dequant_dot(_ptr(w), _ptr(w_scale), _ptr(x), _ptr(x_scale), rows, 4 * kw, batch,
                                    _ptr(out), _ptr(acc), stream), "i8_dequant_dot")
    return (out, acc) if want_acc else out


def packed_dot(fields: torch.Tensor, scales: torch.Tensor, rhs: torch.Tensor, count: int,
               initial: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """fields int32 [records][outputs], scales int16/uint16 binary16 bits [records][outputs],
    rhs f32 [records][streams][4] -> out f32 [outputs] (the pages' ordered packed-dot recurrence)."""
    device, stream = _target(fields, "fields")
    _dev(fields, torch.int32, "fields", device)
    if scales.dtype == torch.float16:
        scales = scales.view(torch.int16)
    if scales.dtype not in (torch.int16, torch.uint16):
        raise TypeError("scales must hold binary16 bit patterns (float16, int16 or uint16)")
    _dev(scales, scales.dtype, "scales", device)
    _dev(rhs, torch.float32, "rhs", device)
    _require(fields.dim() == 2 and fields.is_contiguous(), "fields must be a contiguous [records][outputs] tensor")
    _require(scales.shape == fields.shape and scales.is_contiguous(), "scales must be contiguous, shaped as fields")
    _require(rhs.dim() == 3 and rhs.shape[2] == 4 and rhs.is_contiguous() and rhs.shape[0] >= count,
             "rhs must be a contiguous [records >= count][streams][4] tensor")
    records, outputs = fields.shape
    _buffer(initial, torch.float32, outputs, "initial", device, optional=True)
    if out is None:
        out = torch.empty(outputs, dtype=torch.float32, device=fields.device)
    _buffer(out, torch.float32, outputs, "out", device)
    _check(_lib.loom_packed_dot(_ptr(fields), _ptr(scales), _ptr(rhs), rhs.shape[1], _ptr(initial), records, count,
                                outputs, _ptr(out), stream), "packed_dot")
    return out


def sum_guarded_rows(values: torch.Tensor, count: int, columns: int, active_lanes: int,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """values f32 [rows_alloc][32][4] -> sums f32 [32] (the pages' guarded ragged row sum)."""
    device, stream = _target(values, "values")
    _dev(values, torch.float32, "values", device)
    _require(values.dim() == 3 and tuple(values.shape[1:]) == (32, 4) and values.is_contiguous(),
             "values must be a contiguous [rows][32][4] tensor")
    if out is None:
        out = torch.empty(32, dtype=torch.float32, device=values.device)
    _buffer(out, torch.float32, 32, "out", device)
    _check(_lib.loom_sum_guarded_rows(_ptr(values), values.shape[0], count, columns, active_lanes, _ptr(out),
                                      stream), "sum_guarded_rows")
    return out


def routed_combine(ids: torch.Tensor, weights: torch.Tensor, payload: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """ids int32 [tokens][routes], weights f32 [tokens][routes], payload f32 [num_rows][hidden]
    -> out f32 [tokens][hidden] (routed MoE combine; out-of-range ids are missing routes)."""
    device, stream = _target(ids, "ids")
    _dev(ids, torch.int32, "ids", device)
    _dev(weights, torch.float32, "weights", device)
    _dev(payload, torch.float32, "payload", device)
    _require(ids.dim() == 2 and ids.is_contiguous(), "ids must be a contiguous [tokens][routes] tensor")
    _require(weights.shape == ids.shape and weights.is_contiguous(), "weights must be contiguous, shaped as ids")
    _require(payload.dim() == 2 and payload.is_contiguous(), "payload must be a contiguous [rows][hidden] tensor")
    tokens, routes = ids.shape
    num_rows, hidden = payload.shape
    if out is None:
        out = torch.empty(tokens, hidden, dtype=torch.float32, device=ids.device)
    _buffer(out, torch.float32, tokens * hidden, "out", device)
    _check(_lib.loom_routed_combine(_ptr(ids), _ptr(weights), _ptr(payload), num_rows, tokens, routes, hidden,
                                    _ptr(out), stream), "routed_combine")
    return out


# ------------------------------------------------------------------ int8 feed-forward operators

def _type(dtype, name: str) -> int:
    if dtype not in _TYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return _TYPES[dtype]


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _rows_of(t: torch.Tensor, dtype, rows: int, cols: int, name: str, device: int) -> int:
    """Checks a [rows][cols] matrix with unit column stride and any row stride >= cols; returns the row stride."""
    _dev(t, dtype, name, device)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {list(t.shape)}")
    if rows == 0 or cols == 0:
        return max(cols, 1)
    stride, unit = t.stride()
    if unit != 1 and cols != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows == 1:
        return cols
    if stride < cols:
        raise ValueError(f"{name} has overlapping rows")
    return stride


def _weights(w, w_scale, device, w_name, s_name):
    """Checks packed weights [rows][k/4] and their scales -> (rows, k / 4)."""
    _dev(w, torch.int32, w_name, device)
    if w.dim() != 2 or not w.is_contiguous():
        raise ValueError(f"{w_name} must be a contiguous [rows][k/4] tensor")
    rows, kw = w.shape
    _buffer(w_scale, torch.float32, rows, s_name, device)
    return rows, kw


def _activations(x, x_scale, kw, device, w_name):
    """Checks packed activations [tokens][k/4] or [k/4] and their scales -> tokens."""
    _dev(x, torch.int32, "x", device)
    if x.dim() not in (1, 2) or not x.is_contiguous() or x.shape[-1] != kw:
        raise ValueError(f"x must be a contiguous [tokens][k/4] tensor with the same k as {w_name}")
    tokens = x.shape[0] if x.dim() == 2 else 1
    _buffer(x_scale, torch.float32, tokens, "x_scale", device, optional=True)
    return tokens


def _gated_operands(w_gate, gate_scale, w_up, up_scale, x, x_scale, device):
    """The operands of the gated projection -> (rows, k, tokens)."""
    rows, kw = _weights(w_gate, gate_scale, device, "w_gate", "gate_scale")
    _weights(w_up, up_scale, device, "w_up", "up_scale")
    _require(w_up.shape == w_gate.shape, "w_up must be shaped as w_gate")
    return rows, 4 * kw, _activations(x, x_scale, kw, device, "w_gate")


def _result(out, dtype, tokens, rows, like, device):
    """The output tensor (made here if None) -> (out, loom_type, row stride)."""
    if out is None:
        kind = _type(dtype, "dtype")
        return torch.empty((tokens, rows), dtype=dtype, device=like.device), kind, rows
    kind = _type(getattr(out, "dtype", None), "out")
    return out, kind, _rows_of(out, out.dtype, tokens, rows, "out", device)


def quantize_rows(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """x [rows][cols] f32, f16 or bf16 with unit column stride (any row stride), cols % 4 == 0
    -> (q int32 [rows][cols/4] packed int8, scale f32 [rows]) with x ~ q * scale, |q| <= 127."""
    device, stream = _target(x, "x")
    kind = _type(x.dtype, "x")
    _require(x.dim() == 2, "x must be [rows][cols]")
    rows, cols = x.shape
    stride = _rows_of(x, x.dtype, rows, cols, "x", device)
    _require(cols % 4 == 0, "x must have a multiple of 4 columns")
    if q is None:
        q = torch.empty(rows, cols // 4, dtype=torch.int32, device=x.device)
    _buffer(q, torch.int32, rows * (cols // 4), "q", device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    _buffer(scale, torch.float32, rows, "scale", device)
    _check(_lib.loom_quantize_rows(_ptr(x), kind, rows, cols, stride, _ptr(q), _ptr(scale), stream), "quantize_rows")
    return q, scale


def i8_matmul(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """w int32 [rows][k/4], x int32 [tokens][k/4] or [k/4] (packed int8), w_scale f32 [rows], x_scale f32 [tokens],
    bias f32 [rows] -> out [tokens][rows] of ``dtype`` (or of ``out``, whose rows may be strided)."""
    device, stream = _target(w, "w")
    rows, kw = _weights(w, w_scale, device, "w", "w_scale")
    tokens = _activations(x, x_scale, kw, device, "w")
    _buffer(bias, torch.float32, rows, "bias", device, optional=True)
    out, kind, stride = _result(out, dtype, tokens, rows, w, device)
    _check(_lib.loom_i8_matmul(_ptr(w), _ptr(w_scale), _ptr(x), _ptr(x_scale), _ptr(bias), rows, 4 * kw, tokens,
                               _ptr(out), kind, stride, stream), "i8_matmul")
    return out


def i8_gated_projection(w_gate: torch.Tensor, gate_scale: torch.Tensor, w_up: torch.Tensor, up_scale: torch.Tensor,
                        x: torch.Tensor, x_scale: torch.Tensor | None = None, act: str = "silu",
                        dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x w_gate^T) * (x w_up^T) with the scales of i8_matmul -> out [tokens][rows] of ``dtype`` (or of ``out``).
    act: 'silu', 'gelu', 'gelu_tanh' or 'relu'."""
    device, stream = _target(w_gate, "w_gate")
    rows, k, tokens = _gated_operands(w_gate, gate_scale, w_up, up_scale, x, x_scale, device)
    code = _act(act)
    out, kind, stride = _result(out, dtype, tokens, rows, w_gate, device)
    _check(_lib.loom_i8_gated_projection(_ptr(w_gate), _ptr(gate_scale), _ptr(w_up), _ptr(up_scale), _ptr(x),
                                         _ptr(x_scale), rows, k, tokens, code, _ptr(out), kind, stride, stream),
           "i8_gated_projection")
    return out


def i8_gated_projection_backward_workspace(rows: int, k: int, tokens: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that i8_gated_projection_backward needs for these sizes and this type of gradient."""
    n = ctypes.c_int64()
    _check(_lib.loom_i8_gated_projection_backward_workspace(rows, k, tokens, _type(dtype, "dtype"), ctypes.byref(n)),
           "i8_gated_projection_backward_workspace")
    return n.value


def i8_gated_projection_backward(w_gate: torch.Tensor, gate_scale: torch.Tensor, w_up: torch.Tensor,
                                 up_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None,
                                 d_out: torch.Tensor, act: str = "silu", want_d_x: bool = True,
                                 want_d_scales: bool = True, workspace: torch.Tensor | None = None):
    """Gradients of i8_gated_projection for d_out [tokens][rows] (f32, f16 or bf16, rows may be strided)
    -> (d_x [tokens][k] of d_out's type, d_gate_scale f32 [rows], d_up_scale f32 [rows]).

    d_x is the gradient of the dequantised activation x * x_scale.  A gradient that is not wanted is None.
    workspace: a uint8 buffer of i8_gated_projection_backward_workspace bytes, 16-byte aligned (made here if None)."""
    device, stream = _target(w_gate, "w_gate")
    rows, k, tokens = _gated_operands(w_gate, gate_scale, w_up, up_scale, x, x_scale, device)
    code = _act(act)
    kind = _type(getattr(d_out, "dtype", None), "d_out")
    stride = _rows_of(d_out, d_out.dtype, tokens, rows, "d_out", device)
    need = i8_gated_projection_backward_workspace(rows, k, tokens, d_out.dtype)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=w_gate.device)
    _buffer(workspace, torch.uint8, need, "workspace", device)
    d_x = torch.empty(tokens, k, dtype=d_out.dtype, device=w_gate.device) if want_d_x else None
    d_gate = torch.empty(rows, dtype=torch.float32, device=w_gate.device) if want_d_scales else None
    d_up = torch.empty(rows, dtype=torch.float32, device=w_gate.device) if want_d_scales else None
    _check(_lib.loom_i8_gated_projection_backward(_ptr(w_gate), _ptr(gate_scale), _ptr(w_up), _ptr(up_scale), _ptr(x),
                                                  _ptr(x_scale), rows, k, tokens, code, _ptr(d_out), kind, stride,
                                                  _ptr(d_x), _ptr(d_gate), _ptr(d_up), _ptr(workspace),
                                                  workspace.numel(), stream),
           "i8_gated_projection_backward")
    return d_x, d_gate, d_up


def pack_int8(t: torch.Tensor) -> torch.Tensor:
    """View an int8 [..., k] tensor (k % 4 == 0) as packed int32 [..., k/4] words (no copy)."""
    _require(t.dtype == torch.int8 and t.shape[-1] % 4 == 0 and t.is_contiguous(),
             "pack_int8 needs a contiguous int8 tensor whose last dimension is a multiple of 4")
    if t.shape[-1] == 0:
        return torch.empty(*t.shape[:-1], 0, dtype=torch.int32, device=t.device)
    return t.view(torch.int32)


# ------------------------------------------------------------------ experts with 4-bit weights

def _made(t, dtype, shape, numel, name, like, device):
    """A caller's buffer, checked, or a new tensor of that shape."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _buffer(t, dtype, numel, name, device)


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, got {score!r}")
    return SCORES[score]


def _logits(logits, device):
    """Checks router logits [tokens][experts] -> (loom_type, tokens, experts, row stride)."""
    kind = _type(logits.dtype, "logits")
    _require(logits.dim() == 2, "logits must be [tokens][experts]")
    tokens, experts = logits.shape
    return kind, tokens, experts, _rows_of(logits, logits.dtype, tokens, experts, "logits", device)


def route_experts(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None,
                  groups: int = 1, top_groups: int = 1, group_top: int = 2, renormalize: bool = True,
                  scale: float = 1.0, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None):
    """logits [tokens][experts] f32, f16 or bf16 (rows may be strided) -> (ids int32 [tokens][top_k], weights f32
    [tokens][top_k]): the experts of the largest choices, score + bias (f32 [experts]) or the logit without a bias,
    among the top_groups best of ``groups`` runs of experts, and scale * score, over their sum if renormalize.

    score: 'softmax' or 'sigmoid'.  group_top: how many of a group's largest choices make its value, 1 or 2.
    Experts whose logit is -inf are never chosen; ids that are missing for that are -1, with weight 0."""
    device, stream = _target(logits, "logits")
    kind, tokens, experts, stride = _logits(logits, device)
    code = _score(score)
    _buffer(bias, torch.float32, experts, "bias", device, optional=True)
    shape = (tokens, top_k if 0 < top_k <= 64 else 0)  # more are refused below
    ids = _made(ids, torch.int32, shape, tokens * top_k, "ids", logits, device)
    weights = _made(weights, torch.float32, shape, tokens * top_k, "weights", logits, device)
    _check(_lib.loom_route_experts(_ptr(logits), kind, tokens, experts, stride, code, _ptr(bias), groups, top_groups,
                                   group_top, top_k, int(renormalize), scale, _ptr(ids), _ptr(weights), stream),
           "route_experts")
    return ids, weights


def route_experts_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, score: str = "softmax",
                           renormalize: bool = True, scale: float = 1.0,
                           d_logits: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of route_experts' weights for d_weights f32 [tokens][top_k], with its logits and ids
    -> d_logits [tokens][experts] of the logits' type (rows of a given ``d_logits`` may be strided)."""
    device, stream = _target(logits, "logits")
    kind, tokens, experts, stride = _logits(logits, device)
    code = _score(score)
    _dev(ids, torch.int32, "ids", device)
    _dev(d_weights, torch.float32, "d_weights", device)
    _require(ids.dim() == 2 and ids.shape[0] == tokens and ids.is_contiguous(), "ids must be a contiguous [tokens][top_k] tensor")
    _require(d_weights.shape == ids.shape and d_weights.is_contiguous(), "d_weights must be contiguous, shaped as ids")
    if d_logits is None:
        d_logits, d_stride = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device), experts
    else:
        d_stride = _rows_of(d_logits, logits.dtype, tokens, experts, "d_logits", device)
    _check(_lib.loom_route_experts_backward(_ptr(logits), kind, tokens, experts, stride, code, ids.shape[1],
                                            int(renormalize), scale, _ptr(ids), _ptr(d_weights), _ptr(d_logits),
                                            d_stride, stream), "route_experts_backward")
    return d_logits


def group_routes_workspace(tokens: int, routes: int, experts: int) -> int:
    """Bytes of workspace that group_routes needs for these sizes."""
    n = ctypes.c_int64()
    _check(_lib.loom_group_routes_workspace(tokens, routes, experts, ctypes.byref(n)), "group_routes_workspace")
    return n.value


_group_need = functools.lru_cache(maxsize=256)(group_routes_workspace)  # a function of the sizes alone


def group_routes(ids: torch.Tensor, experts: int, slots: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                 offsets: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """ids int32 [tokens][routes] -> (slots int32 [tokens][routes], rows int32 [tokens * routes], offsets int32
    [experts + 1]): where each route stands in the order of experts (-1: its id is no expert), whose token stands at
    each place (-1 past the last), and where each expert's places begin.

    slots are the ids that routed_combine takes for the rows of the experts' products.
    workspace: a uint8 buffer of group_routes_workspace bytes, 4-byte aligned (made here if None)."""
    device, stream = _target(ids, "ids")
    _dev(ids, torch.int32, "ids", device)
    _require(ids.dim() == 2 and ids.is_contiguous(), "ids must be a contiguous [tokens][routes] tensor")
    tokens, routes = ids.shape
    pairs, need = tokens * routes, _group_need(tokens, routes, experts)
    slots = _made(slots, torch.int32, (tokens, routes), pairs, "slots", ids, device)
    rows = _made(rows, torch.int32, pairs, pairs, "rows", ids, device)
    offsets = _made(offsets, torch.int32, experts + 1, experts + 1, "offsets", ids, device)
    if workspace is not None or need > 0:
        workspace = _made(workspace, torch.uint8, need, need, "workspace", ids, device)
    _check(_lib.loom_group_routes(_ptr(ids), tokens, routes, experts, _ptr(slots), _ptr(rows), _ptr(offsets),
                                  _ptr(workspace), need, stream), "group_routes")
    return slots, rows, offsets


def _weights4(w, w_scale, group, lead, device, w_name, s_name):
    """Checks packed 4-bit weights [rows][k/8] (experts first where lead is 3) and their scales [..][rows][groups]
    -> (k, the scales' loom_type)."""
    _dev(w, torch.int32, w_name, device)
    shape = "[rows][k/8]" if lead == 2 else "[experts][rows][k/8]"
    if w.dim() != lead or not w.is_contiguous():
        raise ValueError(f"{w_name} must be a contiguous {shape} tensor")
    kind = _type(getattr(w_scale, "dtype", None), s_name)
    _require(group >= 1, "group must be positive")
    k = 8 * w.shape[-1]
    count = w.shape[0] * (w.shape[1] if lead == 3 else 1)
    groups = -(-k // group)
    _buffer(w_scale, w_scale.dtype, count * groups, s_name, device)
    # scales of shorter groups are more than enough, and would be read as if they were these
    if w_scale.dim() > 1 and w_scale.shape[-1] != groups:
        raise ValueError(f"{s_name} has {w_scale.shape[-1]} scales a channel, k {k} in groups of {group} needs {groups}")
    return k, kind


def _activations4(x, x_scale, k, device, w_name):
    """Checks packed activations [tokens][k/4] or [k/4] and their scales -> tokens."""
    return _activations(x, x_scale, k // 4, device, w_name)


def i4_matmul(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, group: int = 128, dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """w int32 [rows][k/8] (packed 4-bit, see pack_int4), w_scale f32, f16 or bf16 [rows][ceil(k / group)], x int32
    [tokens][k/4] or [k/4] (packed int8), x_scale f32 [tokens], bias f32 [rows] -> out [tokens][rows] of ``dtype`` (or
    of ``out``, whose rows may be strided).  group: a power of two, at least 32; k % 32 == 0; w and x 16-byte aligned."""
    device, stream = _target(w, "w")
    k, scales = _weights4(w, w_scale, group, 2, device, "w", "w_scale")
    rows = w.shape[0]
    tokens = _activations4(x, x_scale, k, device, "w")
    _buffer(bias, torch.float32, rows, "bias", device, optional=True)
    out, kind, stride = _result(out, dtype, tokens, rows, w, device)
    _check(_lib.loom_i4_matmul(_ptr(w), _ptr(w_scale), scales, group, _ptr(x), _ptr(x_scale), _ptr(bias), rows, k, tokens,
                               _ptr(out), kind, stride, stream), "i4_matmul")
    return out


def _routed(x, x_scale, index, offsets, experts, k, device, w_name):
    """Checks the activations, index and offsets of an experts' product -> (routed rows, rows of x)."""
    x_rows = _activations4(x, x_scale, k, device, w_name)
    _buffer(offsets, torch.int32, experts + 1, "offsets", device)
    if index is None:
        return x_rows, x_rows
    _dev(index, torch.int32, "index", device)
    _require(index.is_contiguous(), "index must be contiguous")
    return index.numel(), x_rows


def i4_expert_matmul(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None,
                     offsets: torch.Tensor, index: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     group: int = 128, dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """i4_matmul for experts: w int32 [experts][rows][k/8], w_scale [experts][rows][ceil(k / group)], bias f32
    [experts][rows]; routed rows offsets[e] .. offsets[e + 1] - 1 (group_routes) are rows index[p] of x (or rows p of x,
    without an index) times the weights of expert e -> out [routed rows][rows].

    Rows of out that belong to no expert are not written: hand in an ``out`` to know what they hold."""
    device, stream = _target(w, "w")
    k, scales = _weights4(w, w_scale, group, 3, device, "w", "w_scale")
    experts, rows = w.shape[:2]
    pairs, x_rows = _routed(x, x_scale, index, offsets, experts, k, device, "w")
    _buffer(bias, torch.float32, experts * rows, "bias", device, optional=True)
    out, kind, stride = _result(out, dtype, pairs, rows, w, device)
    _check(_lib.loom_i4_expert_matmul(_ptr(w), _ptr(w_scale), scales, group, _ptr(x), _ptr(x_scale), x_rows, _ptr(index),
                                      _ptr(offsets), _ptr(bias), experts, rows, k, pairs, _ptr(out), kind, stride,
                                      stream), "i4_expert_matmul")
    return out


def i4_expert_gated_projection(w_gate: torch.Tensor, gate_scale: torch.Tensor, w_up: torch.Tensor,
                               up_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None,
                               offsets: torch.Tensor, index: torch.Tensor | None = None, act: str = "silu",
                               group: int = 128, dtype: torch.dtype = torch.bfloat16,
                               out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x w_gate^T) * (x w_up^T) for experts, operands as in i4_expert_matmul for both weights -> out [routed
    rows][rows].  act: 'silu', 'gelu', 'gelu_tanh' or 'relu'."""
    device, stream = _target(w_gate, "w_gate")
    k, scales = _weights4(w_gate, gate_scale, group, 3, device, "w_gate", "gate_scale")
    _, up_kind = _weights4(w_up, up_scale, group, 3, device, "w_up", "up_scale")
    _require(w_up.shape == w_gate.shape, "w_up must be shaped as w_gate")
    _require(up_kind == scales, "up_scale must have gate_scale's type")
    experts, rows = w_gate.shape[:2]
    pairs, x_rows = _routed(x, x_scale, index, offsets, experts, k, device, "w_gate")
    code = _act(act)
    out, kind, stride = _result(out, dtype, pairs, rows, w_gate, device)
    _check(_lib.loom_i4_expert_gated_projection(_ptr(w_gate), _ptr(gate_scale), _ptr(w_up), _ptr(up_scale), scales, group,
                                                _ptr(x), _ptr(x_scale), x_rows, _ptr(index), _ptr(offsets), experts, rows,
                                                k, pairs, code, _ptr(out), kind, stride, stream),
           "i4_expert_gated_projection")
    return out


def pack_int4(t: torch.Tensor) -> torch.Tensor:
    """int8 values -8 .. 7 [..., k] (k % 32 == 0) as packed int32 [..., k/8] words, on the tensor's own device: of each
    16 bytes, byte b holds element b of 32 in its low four bits and element 16 + b in its high four."""
    _require(t.dtype == torch.int8 and t.shape[-1] % 32 == 0,
             "pack_int4 needs an int8 tensor whose last dimension is a multiple of 32")
    k = t.shape[-1]
    if t.numel() == 0:
        return torch.empty(*t.shape[:-1], k // 8, dtype=torch.int32, device=t.device)
    halves = t.contiguous().view(torch.uint8).view(*t.shape[:-1], k // 32, 2, 16)
    return ((halves[..., 0, :] & 15) | (halves[..., 1, :] << 4)).reshape(*t.shape[:-1], k // 2).view(torch.int32)
