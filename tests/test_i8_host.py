"""Host-side checks of the operators in include/i8_group.h, of the balance loss
and of the 8-bit checkpoint (no GPU): exported symbols, constants, refusals at
the C entry points and in the binding, the references against differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import i8_reference as I
import moe_reference as R
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import i8, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "i8_group.h")).read()
MOE_HEADER = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
FAKE = 0x10000  # never dereferenced: every call below fails a host check first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from nvfp4_block_scaled_group_amd import build
        build.build()
    moe.load_library()
    return i8.load_library()


def test_header_and_binding_name_the_same_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    declared = set(re.findall(r"^(?:int|int64_t)\s+(i8_\w+)\s*\(", text, flags=re.M))
    assert declared == set(i8.EXPORTS)
    for name in declared:
        assert hasattr(lib, name) and callable(getattr(i8, name))


def test_constants_match_the_headers():
    assert int(re.search(r"#define I8_MAX_K (\d+)", HEADER).group(1)) == i8.MAX_K
    assert i8.MAX_K % 16 == 0 and 128 * 128 * i8.MAX_K < 2 ** 31 <= 128 * 128 * (i8.MAX_K + 16)
    assert int(re.search(r"#define MOE_MAX_SEQS (\d+)", MOE_HEADER).group(1)) == moe.MAX_SEQS
    assert int(re.search(r"#define MOE_KEEP8_GROUP (\d+)", MOE_HEADER).group(1)) == moe.KEEP8_GROUP


def with_change(args, at, value):
    out = list(args)
    out[at] = value
    return out


CAST = [FAKE, 100, 64, FAKE, FAKE, None]
CAST_G = [FAKE, 256, 64, 2, FAKE, FAKE, FAKE, FAKE, None]
LINEAR = [FAKE, FAKE, 100, 64, FAKE, FAKE, 32, FAKE, 0, FAKE, 1 << 25, None]
GEMM_G = [FAKE] * 4 + [256, 32, 64, 2, FAKE, FAKE, 0, FAKE, None]
GLU_G = [FAKE] * 4 + [256, 32, 64, 2, FAKE, 0, FAKE, FAKE, None]
TOKEN_GLU = [FAKE, 4, 64, 2, FAKE, FAKE, FAKE, 32, 8, 0, FAKE, None]
TOKEN_LIN = [FAKE, 4, 64, FAKE, FAKE, FAKE, 32, 8, FAKE, None]
BALANCE = [FAKE, 0, 300, 8, 2, FAKE, 0, FAKE, 3, 0.01, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, None]
BALANCE_BWD = [FAKE, 0, 300, 8, 2, 0, FAKE, 3, 0.01, FAKE, FAKE, FAKE, FAKE, FAKE, None]


@pytest.mark.parametrize("fn,args,at,value,status", [
    ("i8_group_cast", CAST, 0, None, -1), ("i8_group_cast", CAST, 1, -1, -1), ("i8_group_cast", CAST, 1, (1 << 24) + 1, -1),
    ("i8_group_cast", CAST, 2, 24, -1), ("i8_group_cast", CAST, 2, 0, -1), ("i8_group_cast", CAST, 2, 131072, -1),
    ("i8_group_cast", CAST, 3, None, -1), ("i8_group_cast", CAST, 4, None, -1), ("i8_group_cast", CAST, 0, FAKE + 8, -3),
    ("i8_group_cast", CAST, 3, FAKE + 8, -3), ("i8_group_cast", CAST, 4, FAKE + 2, -3),
    ("i8_group_cast_graphsafe", CAST_G, 1, 200, -1), ("i8_group_cast_graphsafe", CAST_G, 3, 0, -1),
    ("i8_group_cast_graphsafe", CAST_G, 4, None, -1), ("i8_group_cast_graphsafe", CAST_G, 7, None, -1),
    ("i8_group_cast_graphsafe", CAST_G, 4, FAKE + 2, -3), ("i8_group_cast_graphsafe", CAST_G, 3, 4097, -1),
    ("i8_linear", LINEAR, 0, None, -1), ("i8_linear", LINEAR, 1, None, -1), ("i8_linear", LINEAR, 2, -1, -1),
    ("i8_linear", LINEAR, 3, 72, -1), ("i8_linear", LINEAR, 3, 131072, -1), ("i8_linear", LINEAR, 4, None, -1),
    ("i8_linear", LINEAR, 6, 24, -1), ("i8_linear", LINEAR, 6, 0, -1), ("i8_linear", LINEAR, 6, (1 << 20) + 16, -1),
    ("i8_linear", LINEAR, 7, None, -1), ("i8_linear", LINEAR, 8, 2, -1), ("i8_linear", LINEAR, 0, FAKE + 8, -3),
    ("i8_linear", LINEAR, 4, FAKE + 8, -3), ("i8_linear", LINEAR, 5, FAKE + 1, -3), ("i8_linear", LINEAR, 7, FAKE + 8, -3),
    ("i8_linear", LINEAR, 2, (1 << 24) + 1, -1),
    ("i8_group_gemm_graphsafe", GEMM_G, 4, 200, -1), ("i8_group_gemm_graphsafe", GEMM_G, 5, 40, -1),
    ("i8_group_gemm_graphsafe", GEMM_G, 6, 40, -1), ("i8_group_gemm_graphsafe", GEMM_G, 7, 0, -1),
    ("i8_group_gemm_graphsafe", GEMM_G, 8, None, -1), ("i8_group_gemm_graphsafe", GEMM_G, 9, None, -1),
    ("i8_group_gemm_graphsafe", GEMM_G, 10, 3, -1), ("i8_group_gemm_graphsafe", GEMM_G, 11, None, -1),
    ("i8_group_gemm_graphsafe", GEMM_G, 2, FAKE + 8, -3), ("i8_group_gemm_graphsafe", GEMM_G, 9, FAKE + 8, -3),
    ("i8_group_glu_graphsafe", GLU_G, 5, 24, -1), ("i8_group_glu_graphsafe", GLU_G, 5, (1 << 19) + 16, -1),
    ("i8_group_glu_graphsafe", GLU_G, 9, 2, -1), ("i8_group_glu_graphsafe", GLU_G, 10, None, -1),
    ("i8_group_glu_graphsafe", GLU_G, 10, FAKE + 8, -3), ("i8_group_glu_graphsafe", GLU_G, 11, None, -1),
    ("i8_token_glu", TOKEN_GLU, 2, 40, -1), ("i8_token_glu", TOKEN_GLU, 7, 24, -1), ("i8_token_glu", TOKEN_GLU, 9, 2, -1),
    ("i8_token_glu", TOKEN_GLU, 1, 513, -1), ("i8_token_glu", TOKEN_GLU, 3, 17, -1), ("i8_token_glu", TOKEN_GLU, 4, None, -1),
    ("i8_token_glu", TOKEN_GLU, 5, FAKE + 8, -3), ("i8_token_glu", TOKEN_GLU, 8, 4097, -1),
    ("i8_token_linear", TOKEN_LIN, 1, 1025, -1), ("i8_token_linear", TOKEN_LIN, 6, 8, -1),
    ("i8_token_linear", TOKEN_LIN, 8, None, -1), ("i8_token_linear", TOKEN_LIN, 8, FAKE + 4, -3),
    ("i8_token_linear", TOKEN_LIN, 7, 0, -1), ("i8_token_linear", TOKEN_LIN, 0, FAKE + 8, -3),
    ("moe_balance", BALANCE, 0, None, -1), ("moe_balance", BALANCE, 1, 2, -1), ("moe_balance", BALANCE, 2, -1, -1),
    ("moe_balance", BALANCE, 2, (1 << 23) + 1, -1), ("moe_balance", BALANCE, 3, 0, -1), ("moe_balance", BALANCE, 3, 4097, -1),
    ("moe_balance", BALANCE, 4, 0, -1), ("moe_balance", BALANCE, 4, 9, -1), ("moe_balance", BALANCE, 5, None, -1),
    ("moe_balance", BALANCE, 6, 2, -1), ("moe_balance", BALANCE, 7, None, -1), ("moe_balance", BALANCE, 8, 0, -1),
    ("moe_balance", BALANCE, 8, 65536, -1), ("moe_balance", BALANCE, 10, None, -1), ("moe_balance", BALANCE, 11, None, -1),
    ("moe_balance", BALANCE, 12, None, -1), ("moe_balance", BALANCE, 13, None, -1), ("moe_balance", BALANCE, 14, None, -1),
    ("moe_balance", BALANCE, 15, 64, -1), ("moe_balance", BALANCE, 0, FAKE + 2, -3), ("moe_balance", BALANCE, 7, FAKE + 2, -3),
    ("moe_balance", BALANCE, 14, FAKE + 2, -3),
    ("moe_balance_bwd", BALANCE_BWD, 4, 17, -1), ("moe_balance_bwd", BALANCE_BWD, 6, None, -1),
    ("moe_balance_bwd", BALANCE_BWD, 9, None, -1), ("moe_balance_bwd", BALANCE_BWD, 10, None, -1),
    ("moe_balance_bwd", BALANCE_BWD, 13, None, -1), ("moe_balance_bwd", BALANCE_BWD, 11, FAKE + 2, -3),
    ("moe_balance_bwd", BALANCE_BWD, 12, FAKE + 2, -3), ("moe_balance_bwd", BALANCE_BWD, 13, FAKE + 2, -3),
])
def test_c_entry_points_refuse(lib, fn, args, at, value, status):
    assert getattr(lib, fn)(*with_change(args, at, value)) == status


def test_host_splits_are_checked(lib):
    good, bad = (ctypes.c_int64 * 2)(128, 128), (ctypes.c_int64 * 2)(128, 100)
    ops = [FAKE] * 4
    assert lib.i8_group_gemm(*ops, 228, 32, 64, 2, bad, FAKE, 0, None) == -2
    assert lib.i8_group_gemm(*ops, 384, 32, 64, 2, good, FAKE, 0, None) == -2
    assert lib.i8_group_gemm(*ops, 256, 32, 64, 2, None, FAKE, 0, None) == -1
    assert lib.i8_group_glu(*ops, 228, 32, 64, 2, bad, 0, FAKE, None) == -2
    assert lib.i8_group_glu(*ops, 256, 32, 64, 513, good, 0, FAKE, None) == -1


def test_launches_past_the_limit_are_refused(lib):
    """Tiles that a launch cannot hold."""
    rows = 1 << 24
    sp = (ctypes.c_int64 * 1)(rows)
    assert lib.i8_linear(*with_change(with_change(LINEAR, 2, rows), 6, 1 << 20)) == -1
    assert lib.i8_group_gemm(*[FAKE] * 4, rows, 1 << 20, 64, 1, sp, FAKE, 0, None) == -1
    assert lib.i8_group_glu(*[FAKE] * 4, rows, 1 << 19, 64, 1, sp, 0, FAKE, None) == -1


def test_keep8_entry_points_refuse(lib):
    sp, ops = (ctypes.c_int64 * 2)(128, 128), [FAKE] * 6
    fwd, bwd = lib.moe_glu_keep8, lib.moe_glu_bwd_keep8
    assert fwd(*ops, 256, 24, 128, 2, sp, 0, FAKE, FAKE, FAKE, None) == -1          # f not a multiple of 16
    assert fwd(*ops, 256, 32, 96, 2, sp, 0, FAKE, FAKE, FAKE, None) == -1           # k not a multiple of 128
    assert fwd(*ops, 256, 32, 128, 2, sp, 2, FAKE, FAKE, FAKE, None) == -1          # unknown activation
    assert fwd(*ops, 256, 32, 128, 2, sp, 0, None, FAKE, FAKE, None) == -1
    assert fwd(*ops, 256, 32, 128, 2, sp, 0, FAKE, None, FAKE, None) == -1
    assert fwd(*ops, 256, 32, 128, 2, sp, 0, FAKE, FAKE, None, None) == -1
    assert fwd(*ops, 256, 32, 128, 2, sp, 0, FAKE, FAKE + 8, FAKE, None) == -3
    assert fwd(*ops, 256, 32, 128, 2, sp, 0, FAKE, FAKE, FAKE + 2, None) == -3
    assert fwd(*ops, 228, 32, 128, 2, (ctypes.c_int64 * 2)(128, 100), 0, FAKE, FAKE, FAKE, None) == -2
    assert bwd(*ops, 256, 32, 128, 2, sp, None, FAKE, 0, FAKE, None, None) == -1
    assert bwd(*ops, 256, 32, 128, 2, sp, FAKE, None, 0, FAKE, None, None) == -1
    assert bwd(*ops, 256, 32, 128, 2, sp, FAKE, FAKE, 0, None, None, None) == -1
    assert bwd(*ops, 256, 32, 128, 2, sp, FAKE, FAKE, 0, FAKE, FAKE + 8, None) == -3
    assert bwd(*ops, 256, 32, 128, 2, sp, FAKE + 8, FAKE, 0, FAKE, None, None) == -3
    assert lib.moe_glu_keep8_graphsafe(*ops, 256, 32, 128, 2, None, 0, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_glu_keep8_graphsafe(*ops, 200, 32, 128, 2, FAKE, 0, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_glu_bwd_keep8_graphsafe(*ops, 256, 32, 128, 2, FAKE, FAKE, FAKE, 0, FAKE, None, None, None) == -1


def test_nothing_to_do_is_no_error(lib):
    assert lib.i8_group_cast(*with_change(CAST, 1, 0)) == 0
    assert lib.i8_linear(*with_change(LINEAR, 2, 0)) == 0
    assert lib.i8_group_gemm_graphsafe(*with_change(GEMM_G, 4, 0)) == 0
    assert lib.i8_token_linear(*with_change(TOKEN_LIN, 1, 0)) == 0
    assert lib.moe_balance_bwd(*with_change(BALANCE_BWD, 2, 0)) == 0


def test_balance_workspace_serves_smaller_batches(lib):
    for E in (8, 256, 4096):
        last = 0
        for tokens in sorted({*range(0, 1500, 7), *range(32000, 34000, 13), 65536, 65537, 1 << 20}):
            size = moe.moe_balance_workspace(tokens, E, 3)
            assert last <= size <= (256 + 3) * (8 * E + 4) + 4 * 3 * -(-E // 32) + 4, tokens
            last = size
        assert moe.moe_balance_workspace(4096, E, 3) < moe.moe_balance_workspace(4096, E, 4)
    assert moe.moe_balance_workspace(128, 64, 1) == 0 and moe.moe_balance_workspace(129, 64, 1) > 0
    assert moe.moe_balance_workspace(-1, 64, 1) == -1 and moe.moe_balance_workspace(64, 64, 0) == -1


@pytest.mark.parametrize("k,n", [(16, 16), (2048, 528), (7168, 7168), (5920, 2064), (131056, 256), (4096, 1 << 16)])
def test_linear_workspace_serves_smaller_batches(lib, k, n):
    last = 0
    for rows in sorted({*range(0, 300), *range(300, 9000, 61), 16384, 1 << 20}):
        size = i8.i8_linear_workspace(rows, k, n)
        assert last <= size <= 32 << 20, rows
        last = size
    short = 16 * k <= 200000                                       # few and short rows need none
    assert (i8.i8_linear_workspace(16, k, n) == 0) == short and i8.i8_linear_workspace(17, k, n) > 0


# ------------------------------------------- which kernels the GPU tests reach

FEW, BIG, MID, MID4, MID4_PARTS = 6, 0, 1, 2, 5


@pytest.fixture(scope="module")
def choice():
    import sys
    sys.path.insert(0, os.path.join(ROOT, "tests", "hip"))
    import build_selftest
    if not os.path.exists(build_selftest.CHOICE_LIB):
        build_selftest.build_choice()
    fn = ctypes.CDLL(build_selftest.CHOICE_LIB).i8_choice
    fn.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_void_p]

    def ask(kind, rows, n, k, splits=None, device=False):
        routing = 0 if splits is None else 2 if device else 1
        E, given = (1, None) if splits is None else (len(splits), (ctypes.c_int64 * len(splits))(*splits))
        return fn({"f32": 0, "bf16": 1, "glu": 2}[kind], routing, rows, n, k, E, given)
    return ask


def parameters(test, names):
    return next(m.args[1] for m in test.pytestmark if m.args and m.args[0] == names)


def test_gpu_cases_reach_every_tile_of_a_projection(choice):
    import test_gpu_i8 as T
    for kind in ("f32", "bf16"):
        assert {choice(kind, m, n, k) for m, n, k in T.LINEAR} == {FEW, BIG, MID, MID4, MID4_PARTS}


@pytest.mark.parametrize("kind", ["f32", "bf16", "glu"])
def test_gpu_cases_reach_every_tile_of_the_experts(choice, kind):
    import test_gpu_i8 as T
    assert {choice(kind, sum(s), n, k, s) for s, n, k in T.GROUPS} == {BIG, MID, MID4}
    wide = 1 if kind != "glu" else 2                               # the tests below halve n for the gated block
    small = parameters(T.test_device_routing_writes_the_routed_rows_alone, "splits,spare")
    large = parameters(T.test_device_routing_of_large_tiles, "splits,spare")
    assert {choice(kind, sum(s) + more, 96 // wide, 208, s, device=True) for s, more in small} == {MID}
    n = 2064 if kind != "glu" else 1040
    assert BIG in {choice(kind, sum(s) + more, n, 400, s, device=True) for s, more in large}
    assert {choice(kind, sum(s) + more, n, k, s, device=True) for s, more, n, k in T.DEVICE} == {MID4}


class _NoCalls:
    def __getattr__(self, name):
        def fail(*args, **kwargs):
            raise AssertionError(f"{name} was called although an argument check should have failed")
        return fail


@pytest.fixture
def cpu_device(monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: torch.device("cpu"))
    monkeypatch.setattr(moe, "_device_index", lambda: -2)  # every buffer through the full checks
    for m in (moe, i8):
        monkeypatch.setattr(m, "load_library", lambda *a, **k: _NoCalls())
        monkeypatch.setattr(m, "_stream", lambda *a: None)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def q8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


NV = lambda: (u8(128, 64), u8(128, 8), f32(128), u8(1, 64, 64), u8(1, 64, 8), f32(64), [128])  # noqa: E731
NVB = lambda: (u8(128, 64), u8(128, 8), f32(128), u8(1, 32, 64), u8(1, 32, 8), f32(32), [128])  # noqa: E731

BAD_CALLS = {
    "cast x": (lambda: i8.i8_group_cast(f32(4, 64), q8(4, 64), f32(4)), "x"),
    "cast x order": (lambda: i8.i8_group_cast(b16(64, 4).t(), q8(4, 64), f32(4)), "x"),
    "cast q": (lambda: i8.i8_group_cast(b16(4, 64), u8(4, 64), f32(4)), "q"),
    "cast q shape": (lambda: i8.i8_group_cast(b16(4, 64), q8(4, 32), f32(4)), "q"),
    "cast scale": (lambda: i8.i8_group_cast(b16(4, 64), q8(4, 64), f32(5)), "scale"),
    "cast offs": (lambda: i8.i8_group_cast_graphsafe(b16(128, 64), i32(2).long(), q8(128, 64), f32(128), i32(1)), "d_offs"),
    "linear columns": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(32, 48), f32(32), f32(4, 32)), "columns"),
    "linear a": (lambda: i8.i8_linear(u8(4, 64), f32(4), q8(32, 64), f32(32), f32(4, 32)), "a_q"),
    "linear scale": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(32, 64), f32(31), f32(4, 32)), "b_scale"),
    "linear out": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(32, 64), f32(32), f32(4, 31)), "out"),
    "linear out type": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(32, 64), f32(32), f32(4, 32).double()), "out"),
    "linear b order": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(64, 32).t(), f32(32), f32(4, 32)), "b_q"),
    "linear workspace": (lambda: i8.i8_linear(q8(4, 64), f32(4), q8(32, 64), f32(32), f32(4, 32), f32(64)), "workspace"),
    "gemm splits": (lambda: i8.i8_group_gemm(q8(128, 64), f32(128), q8(2, 32, 64), f32(2, 32), [128], f32(128, 32)), "splits"),
    "gemm status": (lambda: i8.i8_group_gemm_graphsafe(q8(128, 64), f32(128), q8(2, 32, 64), f32(2, 32), i32(2), f32(128, 32),
                                                       f32(1)), "d_status"),
    "glu channels": (lambda: i8.i8_group_glu(q8(128, 64), f32(128), q8(1, 33, 64), f32(1, 33), [128], b16(128, 16)), "channels"),
    "glu h": (lambda: i8.i8_group_glu(q8(128, 64), f32(128), q8(1, 32, 64), f32(1, 32), [128], b16(128, 32)), "h"),
    "token ids": (lambda: i8.i8_token_linear(b16(4, 64), i32(3), q8(2, 32, 64), f32(2, 32), f32(4, 32)), "ids"),
    "token h": (lambda: i8.i8_token_glu(b16(4, 64), i32(4, 2), q8(2, 32, 64), f32(2, 32), b16(8, 32)), "h"),
    "token device": (lambda: i8.i8_token_glu(b16(4, 64), i32(4, 2), q8(2, 32, 64).to("meta"), f32(2, 32), b16(8, 16)), "b_q"),
    "balance counts": (lambda: moe.moe_balance(f32(4, 8), i32(4, 2), f32(1), i32(1, 7), f32(1, 8), i32(1)), "counts"),
    "balance sequences": (lambda: moe.moe_balance(f32(4, 8), i32(4, 2), f32(1), i32(2, 8), f32(2, 8), i32(2)), "one sequence"),
    "balance ends": (lambda: moe.moe_balance(f32(4, 8), i32(4, 2), f32(1), i32(2, 8), f32(2, 8), i32(2), seq_ends=i32(3)), "seq_ends"),
    "balance ends type": (lambda: moe.moe_balance(f32(4, 8), i32(4, 2), f32(1), i32(2, 8), f32(2, 8), i32(2),
                                                  seq_ends=i32(2).long()), "seq_ends"),
    "balance loss": (lambda: moe.moe_balance(f32(4, 8), i32(4, 2), f32(1).double(), i32(1, 8), f32(1, 8), i32(1)), "loss"),
    "balance dlogits": (lambda: moe.moe_balance_bwd(b16(4, 8), i32(1, 8), i32(1), f32(4, 8), topk=2), "dlogits"),
    "balance add": (lambda: moe.moe_balance_bwd(b16(4, 8), i32(1, 8), i32(1), b16(4, 8), topk=2, add=f32(4, 8)), "add"),
    "balance dloss": (lambda: moe.moe_balance_bwd(b16(4, 8), i32(1, 8), i32(1), b16(4, 8), topk=2, dloss=b16(1)), "dloss"),
    "keep8 codes": (lambda: moe.moe_glu_keep8(*NV(), b16(128, 32), u8(128, 64), b16(2, 128)), "gu8"),
    "keep8 scales": (lambda: moe.moe_glu_keep8(*NV(), b16(128, 32), q8(128, 64), b16(128, 2)), "gu_scale"),
    "keep8 scale type": (lambda: moe.moe_glu_keep8(*NV(), b16(128, 32), q8(128, 64), f32(2, 128)), "gu_scale"),
    "keep8 h": (lambda: moe.moe_glu_bwd_keep8(*NVB(), q8(128, 64), b16(2, 128), b16(128, 64), h=b16(128, 16)), "h"),
    "keep8 dgu": (lambda: moe.moe_glu_bwd_keep8(*NVB(), q8(128, 64), b16(2, 128), b16(128, 32)), "dgu"),
}


@pytest.mark.parametrize("name", sorted(BAD_CALLS))
def test_binding_refuses_wrong_buffers(cpu_device, name):
    call, what = BAD_CALLS[name]
    with pytest.raises(ValueError, match=what):
        call()


# --------------------------------------------------------------- references

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_reference_follows_differences(score):
    rng = np.random.default_rng(4)
    T, E, k = 12, 5, 2
    l = rng.standard_normal((T, E))
    l[3, 1], l[5] = -np.inf, -np.inf
    ids = rng.integers(-1, E, (T, k))
    ends = [4, 4, 11]
    loss, _, _, tokens, grad, _ = I.balance(l, ids, ends, score, 0.7, k)
    assert list(tokens) == [4, 0, 6] and loss > 0
    eps = 1e-6
    for t in range(T):
        for e in range(E):
            if not np.isfinite(l[t, e]):
                assert grad[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += eps
            b[t, e] -= eps
            num = (I.balance(a, ids, ends, score, 0.7, k)[0] - I.balance(b, ids, ends, score, 0.7, k)[0]) / (2 * eps)
            assert abs(num - grad[t, e]) < 1e-8
    # all experts alike: the loss is coef
    even = np.arange(8 * k).reshape(8, k) % 4
    assert abs(I.balance(np.zeros((8, 4)), even, None, score, 0.25, k)[0] - 0.25) < 1e-12


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_balance_bounds_notice_lost_rows(score, at):
    """Without the probabilities of one chunk, or of a 32nd of one, probs and the loss leave the GPU test's bounds."""
    from test_gpu_moe_balance import SUMS, make, rel_of
    T, E, k, ends = SUMS[at]
    rng, lt, l, ids = make(T + E + 1, T, E, k, "f32")
    loss, counts, probs, tokens, _, _ = I.balance(l, ids, ends, score, 0.3, k)
    off, loss_off = I.balance_bounds(l, ids, ends, score, 0.3, k, rel_of(l, E))
    p, _, _ = I.probabilities(l, score)
    rows = max(32, -(-T // 256))
    cuts = [T] if ends is None else ends
    for chunk in (1, 100, 150):
        for lost in (rows, max(rows // 32, 1)):
            b = chunk * rows
            s = int(np.searchsorted(cuts, b, side="right"))
            gone = p[b:b + lost].sum(0)
            assert b + lost <= cuts[s]
            assert (gone > 2 * off[s]).any(), (chunk, lost)
            if lost == rows:
                weight = 0.3 / len(cuts) * E / (k * float(tokens[s]) ** 2)
                assert weight * float(counts[s] @ gone) > 2 * loss_off, chunk


def test_cast_reference_is_the_nearest_code():
    rng = np.random.default_rng(1)
    x = R.bf16_round(rng.standard_normal((50, 64)) * np.exp(5 * rng.standard_normal((50, 1))))[0].float().numpy()
    q, s = I.cast(x)
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 1e-4)).all()
