"""Thin ctypes binding of the products in 8-bit integers in ``include/i8_group.h``.

Rows in int8 with a scale for each token times weights in int8 with a scale for
each channel: one projection, grouped by expert, the experts' gated block, and
the forms for single tokens.  Same manner as ``binding`` and ``moe``: every
function has the name of its C entry point, checks its buffers on the host
(ValueError), passes the current stream and raises ``Nvfp4GroupError`` on a
non-zero status.  Outputs are the caller's.

The experts of a layer on packed rows (weights cast once, a channel to a row)::

    i8_group_cast(w.view(E * n, k), w_q.view(E * n, k), w_scale.view(-1))
    i8_group_cast_graphsafe(packed, offs, x_q, x_scale, status)
    i8_group_glu_graphsafe(x_q, x_scale, gate_up_q, gate_up_scale, offs, h, status)
    i8_group_cast_graphsafe(h, offs, h_q, h_scale, status)
    i8_group_gemm_graphsafe(h_q, h_scale, down_q, down_scale, offs, y, status)
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .binding import F32, I32, U8, _check
from .moe import (ACT_GELU, ACT_SILU, B16, I8, MOE_BF16, MOE_F32, _buf, _dims, _exact,  # noqa: F401
                  _host_splits, _routing, _stream)

MAX_K = 131056
OUT = F32 + B16

EXPORTS = (
    "i8_group_cast", "i8_group_cast_graphsafe", "i8_linear_workspace", "i8_linear", "i8_group_gemm",
    "i8_group_gemm_graphsafe", "i8_group_glu", "i8_group_glu_graphsafe", "i8_token_glu", "i8_token_linear",
)

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_lib = None


def load_library() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    L = _b.load_library()
    L.i8_group_cast.argtypes = [_P, _I64, _I64, _P, _P, _P]
    L.i8_group_cast_graphsafe.argtypes = [_P, _I64, _I64, _I32, _P, _P, _P, _P, _P]
    L.i8_linear_workspace.argtypes = [_I64, _I64, _I64]
    L.i8_linear.argtypes = [_P, _P, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _I64, _P]
    L.i8_group_gemm.argtypes = [_P] * 4 + [_I64, _I64, _I64, _I32, _P, _P, _I32, _P]
    L.i8_group_gemm_graphsafe.argtypes = [_P] * 4 + [_I64, _I64, _I64, _I32, _P, _P, _I32, _P, _P]
    L.i8_group_glu.argtypes = [_P] * 4 + [_I64, _I64, _I64, _I32, _P, _I32, _P, _P]
    L.i8_group_glu_graphsafe.argtypes = [_P] * 4 + [_I64, _I64, _I64, _I32, _P, _I32, _P, _P, _P]
    L.i8_token_glu.argtypes = [_P, _I64, _I64, _I32, _P, _P, _P, _I64, _I32, _I32, _P, _P]
    L.i8_token_linear.argtypes = [_P, _I64, _I64, _P, _P, _P, _I64, _I32, _P, _P]
    for name in EXPORTS:
        getattr(L, name).restype = ctypes.c_int64 if name.endswith("_workspace") else ctypes.c_int
    _lib = L
    return L


def _rows(a_q, a_scale):
    m, k = _dims("a_q", a_q, 2)
    return (_buf("a_q", a_q, I8, m * k, True), _exact("a_scale", a_scale, F32, (m,))), m, k


def _channels(b_q, b_scale, k, dim):
    shape = _dims("b_q", b_q, dim)
    if shape[-1] != k:
        raise ValueError(f"b_q has {shape[-1]} columns per channel, the rows have {k}")
    return (_buf("b_q", b_q, I8, 0, True), _exact("b_scale", b_scale, F32, shape[:-1])), shape


def _product(out, m, n):
    """Output [m, n] of a product: f32, or bf16 (raw 16-bit too)."""
    return _exact("out", out, OUT, (m, n)), MOE_F32 if out.dtype == torch.float32 else MOE_BF16


def _cast_buffers(x, q, scale):
    m, k = _dims("x", x, 2)
    return (_buf("x", x, B16, m * k, True), m, k), (_exact("q", q, I8, (m, k)), _exact("scale", scale, F32, (m,)))


def i8_group_cast(x, q, scale, stream=None):
    """x [rows, k] bf16 -> q [rows, k] i8, scale [rows] f32."""
    given, made = _cast_buffers(x, q, scale)
    _check("i8_group_cast", load_library().i8_group_cast(*given, *made, _stream(stream)))


def i8_group_cast_graphsafe(x, d_offs, q, scale, d_status, stream=None):
    """The rows below d_offs[E - 1] of x [m_capacity, k]; the others are neither read nor written."""
    given, made = _cast_buffers(x, q, scale)
    E, = _dims("d_offs", d_offs, 1)
    do, ds = _routing(E, d_offs, d_status)
    _check("i8_group_cast_graphsafe", load_library().i8_group_cast_graphsafe(*given, E, do, *made, ds, _stream(stream)))


def i8_linear_workspace(rows: int, k: int, n: int) -> int:
    """Bytes of workspace that i8_linear needs."""
    return int(load_library().i8_linear_workspace(int(rows), int(k), int(n)))


def i8_linear(a_q, a_scale, b_q, b_scale, out, workspace=None, stream=None):
    """a_q [rows, k] i8, a_scale [rows] times b_q [n, k], b_scale [n] -> out [rows, n] f32 or bf16."""
    a, m, k = _rows(a_q, a_scale)
    b, (n, _) = _channels(b_q, b_scale, k, 2)
    _check("i8_linear", load_library().i8_linear(
        *a, m, k, *b, n, *_product(out, m, n), _buf("workspace", workspace, U8, 0),
        0 if workspace is None else workspace.numel(), _stream(stream)))


def i8_group_gemm(a_q, a_scale, b_q, b_scale, h_splits, out, stream=None):
    """Packed rows a_q [sum_m, k] times their expert's b_q [E, n, k] -> out [sum_m, n] f32 or bf16."""
    a, m, k = _rows(a_q, a_scale)
    b, (E, n, _) = _channels(b_q, b_scale, k, 3)
    _check("i8_group_gemm", load_library().i8_group_gemm(
        *a, *b, m, n, k, E, _host_splits(h_splits, E), *_product(out, m, n), _stream(stream)))


def i8_group_gemm_graphsafe(a_q, a_scale, b_q, b_scale, d_offs, out, d_status, stream=None):
    a, m, k = _rows(a_q, a_scale)
    b, (E, n, _) = _channels(b_q, b_scale, k, 3)
    do, ds = _routing(E, d_offs, d_status)
    _check("i8_group_gemm_graphsafe", load_library().i8_group_gemm_graphsafe(
        *a, *b, m, n, k, E, do, *_product(out, m, n), ds, _stream(stream)))


def _glu_operands(a_q, a_scale, b_q, b_scale, h):
    a, m, k = _rows(a_q, a_scale)
    b, (E, n, _) = _channels(b_q, b_scale, k, 3)
    if n % 2:
        raise ValueError("b_q must hold the gate channels and as many up channels")
    return (*a, *b, m, n // 2, k, E), _exact("h", h, B16, (m, n // 2))


def i8_group_glu(a_q, a_scale, b_q, b_scale, h_splits, h, act=ACT_SILU, stream=None):
    """Packed rows a_q [sum_m, k] and b_q [E, 2f, k], gate channels first -> h = act(g) * u, [sum_m, f] bf16."""
    ops, hp = _glu_operands(a_q, a_scale, b_q, b_scale, h)
    _check("i8_group_glu", load_library().i8_group_glu(*ops, _host_splits(h_splits, ops[-1]), int(act), hp,
                                                       _stream(stream)))


def i8_group_glu_graphsafe(a_q, a_scale, b_q, b_scale, d_offs, h, d_status, act=ACT_SILU, stream=None):
    ops, hp = _glu_operands(a_q, a_scale, b_q, b_scale, h)
    do, ds = _routing(ops[-1], d_offs, d_status)
    _check("i8_group_glu_graphsafe", load_library().i8_group_glu_graphsafe(*ops, do, int(act), hp, ds,
                                                                           _stream(stream)))


def i8_token_glu(x, ids, b_q, b_scale, h, act=ACT_SILU, stream=None):
    """x [T, k] bf16, ids [T, topk] i32, b_q [E, 2f, k] -> h [T * topk, f] bf16."""
    T, k = _dims("x", x, 2)
    topk = _dims("ids", ids, 2)[1]
    b, (E, n, _) = _channels(b_q, b_scale, k, 3)
    if n % 2:
        raise ValueError("b_q must hold the gate channels and as many up channels")
    _check("i8_token_glu", load_library().i8_token_glu(
        _buf("x", x, B16, T * k, True), T, k, topk, _exact("ids", ids, I32, (T, topk)), *b, n // 2, E, int(act),
        _exact("h", h, B16, (T * topk, n // 2)), _stream(stream)))


def i8_token_linear(x, ids, b_q, b_scale, out, stream=None):
    """x [pairs, k] bf16, ids (pairs of them) i32, b_q [E, n, k] -> out [pairs, n] f32."""
    pairs, k = _dims("x", x, 2)
    b, (E, n, _) = _channels(b_q, b_scale, k, 3)
    if not isinstance(ids, torch.Tensor) or ids.numel() != pairs:
        raise ValueError(f"ids must hold one expert for each of the {pairs} rows of x")
    _check("i8_token_linear", load_library().i8_token_linear(
        _buf("x", x, B16, pairs * k, True), pairs, k, _buf("ids", ids, I32, pairs, True), *b, n, E,
        _exact("out", out, F32, (pairs, n)), _stream(stream)))


# ------------------------------------------------------------------ helpers

def alloc_cast(rows: int, k: int, device="cuda"):
    """Buffers of i8_group_cast: q, scale."""
    return {"q": torch.empty((rows, k), dtype=torch.int8, device=device),
            "scale": torch.empty(rows, dtype=torch.float32, device=device)}
