"""Thin ctypes binding of the operators in ``include/moe_ops.h``.

Routing of tokens to experts, movement of rows into and out of the packed
128-row groups, the experts' gated feed-forward block with its backward pass
and its single-token form, and low-rank adapters beside a shared projection.
Same manner as ``binding``: every function has the name of its C entry point,
checks its buffers on the host (ValueError), passes the current stream and
raises ``Nvfp4GroupError`` on a non-zero status.  Outputs are the caller's.

A training step of an expert layer::

    moe_route(logits, ids, weights)                       # [T, E] -> [T, k]
    moe_plan(ids, offs, counts, rows, src, status, workspace)
    moe_dispatch(x, rows, src, offs, packed)              # [T, H] -> [capacity, H]
    ...cast packed (binding.nvfp4_group_quantize_graphsafe)...
    moe_glu_graphsafe(*packed_nvfp4, *gate_up_nvfp4, offs, h, status, gu=gu)
    ...cast h, down projection (binding.nvfp4_group_gemm_graphsafe)...
    moe_combine(y, rows, out, weights=weights)            # [capacity, H] -> [T, H]
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .binding import F32, I32, U8, Nvfp4GroupError, _check, _splits  # noqa: F401

MOE_F32, MOE_BF16 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_SILU, ACT_GELU = 0, 1
MAX_EXPERTS = 4096
MAX_TOPK = 16
MAX_PAIRS = 1 << 24
MAX_TOKEN_PAIRS = 1024
MAX_RANK = 128

EXPORTS = (
    "moe_route", "moe_route_bwd", "moe_plan_workspace", "moe_plan", "moe_dispatch", "moe_combine",
    "moe_glu", "moe_glu_graphsafe", "moe_glu_bwd", "moe_glu_bwd_graphsafe", "moe_token_glu", "moe_token_linear",
    "lora_workspace", "lora_linear",
)

B16 = (torch.bfloat16, torch.int16, torch.uint16)
_P, _I64, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_NVFP4 = [_P, _P, _P]                                   # data, scale, amax
_lib = None


def load_library() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    L = _b.load_library()
    L.moe_route.argtypes = [_P, _I32, _I64, _I32, _I32, _P, _I32, _I32, _F, _P, _P, _P]
    L.moe_route_bwd.argtypes = [_P, _I32, _I64, _I32, _I32, _P, _P, _I32, _I32, _F, _P, _P]
    L.moe_plan_workspace.argtypes = [_I64, _I32]
    L.moe_plan.argtypes = [_P, _I64, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P]
    L.moe_dispatch.argtypes = [_P, _I64, _I64, _I32, _P, _P, _P, _I32, _I64, _P, _P, _I32, _P, _P, _P]
    L.moe_combine.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _P, _P]
    L.moe_glu.argtypes = _NVFP4 * 2 + [_I64, _I64, _I64, _I32, _P, _I32, _P, _P, _P]
    L.moe_glu_graphsafe.argtypes = _NVFP4 * 2 + [_I64, _I64, _I64, _I32, _P, _I32, _P, _P, _P, _P]
    L.moe_glu_bwd.argtypes = _NVFP4 * 2 + [_I64, _I64, _I64, _I32, _P, _P, _I32, _P, _P]
    L.moe_glu_bwd_graphsafe.argtypes = _NVFP4 * 2 + [_I64, _I64, _I64, _I32, _P, _P, _I32, _P, _P, _P]
    L.moe_token_glu.argtypes = [_P, _I64, _I64, _I32, _P] + _NVFP4 + [_I64, _I32, _I32, _P, _P]
    L.moe_token_linear.argtypes = [_P, _I64, _I64, _P] + _NVFP4 + [_I64, _I32, _P, _P]
    L.lora_workspace.argtypes = [_I64, _I64, _I64, _I32]
    L.lora_linear.argtypes = [_P, _I64, _I64] + _NVFP4 + [_I64, _P, _P, _P, _I32, _I32, _P, _P, _P, _I64, _P]
    for name in EXPORTS:
        getattr(L, name).restype = ctypes.c_int64 if name.endswith("_workspace") else ctypes.c_int
    _lib = L
    return L


# the current device's index without the Python layers of torch.cuda (these
# calls sit in decoding loops; a CUDA tensor has initialised the runtime)
_device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream):
    if stream is None and _b._raw_current_stream is not None:
        return _b._raw_current_stream(_device_index())
    return _b._stream(stream)


def _buf(name, t, dtypes, numel, required=False):
    """Address of a caller buffer that passes the binding's checks.  The usual
    case is settled in one expression; anything else goes through
    binding._buf, which names what is wrong."""
    if (type(t) is torch.Tensor and t.dtype in dtypes and t.numel() >= numel and t.is_contiguous()
            and t.get_device() == _device_index()):
        return t.data_ptr()
    return _b._buf(name, t, dtypes, numel, required)


def _routing(e, d_offs, d_status):
    return _buf("d_offs", d_offs, I32, max(e, 1), True), _buf("d_status", d_status, I32, 1, True)


def _dims(name: str, t, dim: int):
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D tensor")
    return t.shape


def _shape(name: str, t, want):
    """A tensor argument whose whole shape is fixed by the others."""
    if not isinstance(t, torch.Tensor) or t.shape != want:
        got = tuple(t.shape) if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name} must be a tensor of shape {tuple(want)}, got {got}")


def _logits(logits):
    T, E = _dims("logits", logits, 2)
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits has dtype {logits.dtype}, expected torch.float32 or torch.bfloat16")
    return _buf("logits", logits, (logits.dtype,), T * E, True), MOE_F32 if logits.dtype == torch.float32 else MOE_BF16, T, E


def _results(name, y):
    """Expert results [rows, width]: fp32, or bf16 (raw 16-bit too)."""
    m, width = _dims(name, y, 2)
    return _buf(name, y, F32 + B16, m * width, True), MOE_F32 if y.dtype == torch.float32 else MOE_BF16, m, width


# ----------------------------------------------------------------- routing

def moe_route(logits, ids, weights, *, select_bias=None, score=SCORE_SOFTMAX, normalize=True, scale=1.0, stream=None):
    """logits [T, E] f32 or bf16 -> ids [T, k] i32 (-1: none), weights [T, k] f32."""
    lp, lt, T, E = _logits(logits)
    k = _dims("ids", ids, 2)[1]
    _shape("ids", ids, (T, k))
    _shape("weights", weights, (T, k))
    _check("moe_route", load_library().moe_route(
        lp, lt, T, E, k, _buf("select_bias", select_bias, F32, E), int(score), int(bool(normalize)), float(scale),
        _buf("ids", ids, I32, T * k, True), _buf("weights", weights, F32, T * k, True), _stream(stream)))


def moe_route_bwd(logits, ids, dweights, dlogits, *, score=SCORE_SOFTMAX, normalize=True, scale=1.0, stream=None):
    """Gradient of moe_route's weights: dweights [T, k] f32 -> dlogits [T, E] in the type of logits."""
    lp, lt, T, E = _logits(logits)
    k = _dims("ids", ids, 2)[1]
    _shape("ids", ids, (T, k))
    _shape("dweights", dweights, (T, k))
    _shape("dlogits", dlogits, (T, E))
    _check("moe_route_bwd", load_library().moe_route_bwd(
        lp, lt, T, E, k, _buf("ids", ids, I32, T * k, True), _buf("dweights", dweights, F32, T * k, True), int(score),
        int(bool(normalize)), float(scale), _buf("dlogits", dlogits, (logits.dtype,), T * E, True), _stream(stream)))


def moe_plan_workspace(pairs: int, num_experts: int) -> int:
    """Bytes of workspace that moe_plan needs for ``pairs`` = tokens * k choices."""
    return int(load_library().moe_plan_workspace(int(pairs), int(num_experts)))


def moe_plan(ids, d_offs, counts, rows, src, d_status, workspace=None, stream=None):
    """ids (any shape) -> d_offs [E], counts [E], rows (ids' shape), src [m_capacity], all i32."""
    if not isinstance(ids, torch.Tensor) or not isinstance(src, torch.Tensor):
        raise ValueError("ids and src must be torch tensors")
    E, = _dims("d_offs", d_offs, 1)
    n, cap = ids.numel(), src.numel()
    _shape("rows", rows, ids.shape)
    _check("moe_plan", load_library().moe_plan(
        _buf("ids", ids, I32, n, True), n, E, cap, _buf("d_offs", d_offs, I32, E, True),
        _buf("counts", counts, I32, E, True), _buf("rows", rows, I32, n, True), _buf("src", src, I32, cap, True),
        _buf("d_status", d_status, I32, 1, True), _buf("workspace", workspace, U8, 0),
        0 if workspace is None else workspace.numel(), _stream(stream)))


def moe_dispatch(x, rows, src, d_offs, out, weights=None, y=None, dweights=None, stream=None):
    """x [T, H] bf16 -> out [m_capacity, H] bf16 at rows [T, k]; with weights [T, k] scaled, with y [m_capacity, H]
    also dweights [T, k] (the gradient of moe_combine)."""
    T, H = _dims("x", x, 2)
    k = _dims("rows", rows, 2)[1]
    _shape("rows", rows, (T, k))
    E, = _dims("d_offs", d_offs, 1)
    cap = _dims("out", out, 2)[0]
    _shape("out", out, (cap, H))
    _shape("src", src, (cap,))
    yp, yt = None, MOE_F32
    if (y is None) != (dweights is None):
        raise ValueError("y and dweights go together")
    if weights is not None:
        _shape("weights", weights, (T, k))
    if y is not None:
        _shape("y", y, (cap, H))
        _shape("dweights", dweights, (T, k))
        yp, yt, _, _ = _results("y", y)
    _check("moe_dispatch", load_library().moe_dispatch(
        _buf("x", x, B16, T * H, True), T, H, k, _buf("rows", rows, I32, T * k, True), _buf("src", src, I32, cap, True),
        _buf("d_offs", d_offs, I32, E, True), E, cap, _buf("weights", weights, F32, T * k), yp, yt,
        _buf("out", out, B16, cap * H, True), _buf("dweights", dweights, F32, T * k), _stream(stream)))


def moe_combine(y, rows, out, weights=None, stream=None):
    """y [m_capacity, H] f32 or bf16 at rows [T, k] -> out [T, H] bf16, weighted by weights [T, k] if given."""
    yp, yt, cap, H = _results("y", y)
    T, k = _dims("rows", rows, 2)
    _shape("out", out, (T, H))
    if weights is not None:
        _shape("weights", weights, (T, k))
    _check("moe_combine", load_library().moe_combine(
        yp, yt, cap, T, H, k, _buf("rows", rows, I32, T * k, True), _buf("weights", weights, F32, T * k),
        _buf("out", out, B16, T * H, True), _stream(stream)))


# ------------------------------------------------- gated feed-forward block

def _rows_operand(a_data, a_scale, a_amax):
    m, half_k = _dims("a_data", a_data, 2)
    k = 2 * half_k
    return (_buf("a_data", a_data, U8, m * half_k, True), _buf("a_scale", a_scale, U8, m * k // 16, True),
            _buf("a_amax", a_amax, F32, m, True)), m, k


def _expert_operand(b_data, b_scale, b_amax, k, what="b"):
    E, n, half_k = _dims(f"{what}_data", b_data, 3)
    if 2 * half_k != k:
        raise ValueError(f"{what}_data has {2 * half_k} columns per line, the rows have {k}")
    return (_buf(f"{what}_data", b_data, U8, E * n * half_k, True),
            _buf(f"{what}_scale", b_scale, U8, E * n * k // 16, True),
            _buf(f"{what}_amax", b_amax, F32, E * n, True)), E, n


def _glu_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax):
    a, m, k = _rows_operand(a_data, a_scale, a_amax)
    b, E, n = _expert_operand(b_data, b_scale, b_amax, k)
    if n % 2:
        raise ValueError("b_data must hold the gate lines and as many up lines")
    return a + b, m, E, n // 2, k


def _host_splits(h_splits, E):
    sp, e = _splits(h_splits)
    if e != E:
        raise ValueError(f"{e} splits for {E} expert operands")
    return sp


def moe_glu(a_data, a_scale, a_amax, b_data, b_scale, b_amax, h_splits, h, gu=None, act=ACT_SILU, stream=None):
    """a: packed rows [sum_m, k/2]; b: [E, 2f, k/2], gate lines first -> h [sum_m, f] bf16 (gu [sum_m, 2f] bf16)."""
    ptrs, m, E, f, k = _glu_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax)
    _check("moe_glu", load_library().moe_glu(
        *ptrs, m, f, k, E, _host_splits(h_splits, E), int(act), _buf("h", h, B16, m * f, True),
        _buf("gu", gu, B16, 2 * m * f), _stream(stream)))


def moe_glu_graphsafe(a_data, a_scale, a_amax, b_data, b_scale, b_amax, d_offs, h, d_status, gu=None, act=ACT_SILU,
                      stream=None):
    ptrs, m, E, f, k = _glu_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax)
    do, ds = _routing(E, d_offs, d_status)
    _check("moe_glu_graphsafe", load_library().moe_glu_graphsafe(
        *ptrs, m, f, k, E, do, int(act), _buf("h", h, B16, m * f, True), _buf("gu", gu, B16, 2 * m * f), ds,
        _stream(stream)))


def _glu_bwd_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax, gu, dgu):
    a, m, k = _rows_operand(a_data, a_scale, a_amax)
    b, E, f = _expert_operand(b_data, b_scale, b_amax, k)
    return a + b, m, E, f, k, _buf("gu", gu, B16, 2 * m * f, True), _buf("dgu", dgu, B16, 2 * m * f, True)


def moe_glu_bwd(a_data, a_scale, a_amax, b_data, b_scale, b_amax, h_splits, gu, dgu, act=ACT_SILU, stream=None):
    """a: gradient of the block's output [sum_m, k/2]; b: down projection as [E, f, k/2] lines; gu [sum_m, 2f] from
    moe_glu -> dgu [sum_m, 2f] bf16."""
    ptrs, m, E, f, k, gp, dp = _glu_bwd_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax, gu, dgu)
    _check("moe_glu_bwd", load_library().moe_glu_bwd(
        *ptrs, m, f, k, E, _host_splits(h_splits, E), gp, int(act), dp, _stream(stream)))


def moe_glu_bwd_graphsafe(a_data, a_scale, a_amax, b_data, b_scale, b_amax, d_offs, gu, dgu, d_status, act=ACT_SILU,
                          stream=None):
    ptrs, m, E, f, k, gp, dp = _glu_bwd_operands(a_data, a_scale, a_amax, b_data, b_scale, b_amax, gu, dgu)
    do, ds = _routing(E, d_offs, d_status)
    _check("moe_glu_bwd_graphsafe", load_library().moe_glu_bwd_graphsafe(
        *ptrs, m, f, k, E, do, gp, int(act), dp, ds, _stream(stream)))


def moe_token_glu(x, ids, b_data, b_scale, b_amax, h, act=ACT_SILU, stream=None):
    """x [T, k] bf16, ids [T, topk] i32, b as in moe_glu -> h [T * topk, f] bf16."""
    T, k = _dims("x", x, 2)
    topk = _dims("ids", ids, 2)[1]
    _shape("ids", ids, (T, topk))
    b, E, n = _expert_operand(b_data, b_scale, b_amax, k)
    if n % 2:
        raise ValueError("b_data must hold the gate lines and as many up lines")
    _check("moe_token_glu", load_library().moe_token_glu(
        _buf("x", x, B16, T * k, True), T, k, topk, _buf("ids", ids, I32, T * topk, True), *b, n // 2, E, int(act),
        _buf("h", h, B16, T * topk * (n // 2), True), _stream(stream)))


def moe_token_linear(x, ids, b_data, b_scale, b_amax, out, stream=None):
    """x [pairs, k] bf16, ids (pairs of them) i32, b [E, n, k/2] -> out [pairs, n] f32."""
    pairs, k = _dims("x", x, 2)
    b, E, n = _expert_operand(b_data, b_scale, b_amax, k)
    if not isinstance(ids, torch.Tensor) or ids.numel() != pairs:
        raise ValueError(f"ids must hold one expert for each of the {pairs} rows of x")
    _check("moe_token_linear", load_library().moe_token_linear(
        _buf("x", x, B16, pairs * k, True), pairs, k, _buf("ids", ids, I32, pairs, True), *b, n, E,
        _buf("out", out, F32, pairs * n, True), _stream(stream)))


# ----------------------------------------------------------------- adapters

def lora_workspace(tokens: int, k: int, n: int, rank: int) -> int:
    """Bytes of workspace that lora_linear needs for up to ``tokens`` rows and ranks up to ``rank`` (0: no adapters)."""
    return int(load_library().lora_workspace(int(tokens), int(k), int(n), int(rank)))


def lora_linear(x, w_data, w_scale, w_amax, lora_a, lora_b, adapter_ids, alpha, y, workspace, stream=None):
    """x [T, k] bf16 times the NVFP4 projection w [n, k/2], plus row t's adapter (adapter_ids[t], -1: none):
    lora_a [A, r, k], lora_b [A, n, r] bf16, alpha [A] f32 -> y [T, n] bf16."""
    T, k = _dims("x", x, 2)
    n, half_k = _dims("w_data", w_data, 2)
    if 2 * half_k != k:
        raise ValueError(f"w_data has {2 * half_k} columns per line, x has {k}")
    A, r, _ = _dims("lora_a", lora_a, 3)
    _shape("lora_a", lora_a, (A, r, k))
    _shape("lora_b", lora_b, (A, n, r))
    _shape("alpha", alpha, (A,))
    _shape("adapter_ids", adapter_ids, (T,))
    _shape("y", y, (T, n))
    _check("lora_linear", load_library().lora_linear(
        _buf("x", x, B16, T * k, True), T, k, _buf("w_data", w_data, U8, n * half_k, True),
        _buf("w_scale", w_scale, U8, n * k // 16, True), _buf("w_amax", w_amax, F32, n, True), n,
        _buf("lora_a", lora_a, B16, A * r * k, True), _buf("lora_b", lora_b, B16, A * n * r, True),
        _buf("alpha", alpha, F32, A, True), A, r, _buf("adapter_ids", adapter_ids, I32, T, True),
        _buf("y", y, B16, T * n, True), _buf("workspace", workspace, U8, 0),
        0 if workspace is None else workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------ helpers

def moe_capacity(tokens: int, topk: int, num_experts: int) -> int:
    """Packed rows that any choice of ``topk`` experts for ``tokens`` tokens fits in (a multiple of 128)."""
    n = int(tokens) * int(topk)
    return min(n * 128, (n + int(num_experts) * 127) // 128 * 128)


def alloc_plan(tokens: int, topk: int, num_experts: int, m_capacity: int | None = None, device="cuda"):
    """Buffers of moe_plan, in the order of its arguments after ids (status zeroed)."""
    cap = moe_capacity(tokens, topk, num_experts) if m_capacity is None else int(m_capacity)
    i32 = dict(dtype=torch.int32, device=device)
    return {"d_offs": torch.empty(num_experts, **i32), "counts": torch.empty(num_experts, **i32),
            "rows": torch.empty((tokens, topk), **i32), "src": torch.empty(cap, **i32),
            "d_status": torch.zeros(1, **i32),
            "workspace": torch.empty(moe_plan_workspace(tokens * topk, num_experts), dtype=torch.uint8, device=device)}
