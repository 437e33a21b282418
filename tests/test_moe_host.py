"""Host-side checks of the operators in include/moe_ops.h (no GPU): exported
symbols, constants, refusals at the C entry points and in the binding."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import moe_reference as R
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
FAKE = 0x10000  # never dereferenced: every call below fails a host check first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from nvfp4_block_scaled_group_amd import build
        build.build()
    return moe.load_library()


def test_header_and_binding_name_the_same_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    declared = set(re.findall(r"^(?:int|int64_t)\s+((?:moe|lora)_\w+)\s*\(", text, flags=re.M))
    assert declared == set(moe.EXPORTS)
    for name in declared:
        assert hasattr(lib, name) and callable(getattr(moe, name))


def test_constants_match_the_header():
    for macro, value in (("MOE_MAX_EXPERTS", moe.MAX_EXPERTS), ("MOE_MAX_TOPK", moe.MAX_TOPK),
                         ("MOE_MAX_TOKEN_PAIRS", moe.MAX_TOKEN_PAIRS), ("LORA_MAX_RANK", moe.MAX_RANK),
                         ("MOE_F32", moe.MOE_F32), ("MOE_BF16", moe.MOE_BF16),
                         ("MOE_SCORE_SOFTMAX", moe.SCORE_SOFTMAX), ("MOE_SCORE_SIGMOID", moe.SCORE_SIGMOID),
                         ("MOE_ACT_SILU", moe.ACT_SILU), ("MOE_ACT_GELU", moe.ACT_GELU)):
        assert int(re.search(rf"#define {macro} (\d+)", HEADER).group(1)) == value
    assert "#define MOE_MAX_PAIRS (1 << 24)" in HEADER and moe.MAX_PAIRS == 1 << 24


def with_change(args, at, value):
    out = list(args)
    out[at] = value
    return out


ROUTE = [FAKE, 0, 4, 8, 2, None, 0, 1, 1.0, FAKE, FAKE, None]
ROUTE_BWD = [FAKE, 0, 4, 8, 2, FAKE, FAKE, 0, 1, 1.0, FAKE, None]
PLAN = [FAKE, 50000, 8, 8192, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, None]
DISPATCH = [FAKE, 4, 64, 2, FAKE, FAKE, FAKE, 8, 256, None, None, 0, FAKE, None, None]
COMBINE = [FAKE, 0, 256, 4, 64, 2, FAKE, None, FAKE, None]
TOKEN_GLU = [FAKE, 4, 64, 2, FAKE, FAKE, FAKE, FAKE, 32, 8, 0, FAKE, None]
TOKEN_LIN = [FAKE, 4, 64, FAKE, FAKE, FAKE, FAKE, 32, 8, FAKE, None]
LORA = [FAKE, 4, 64, FAKE, FAKE, FAKE, 32, FAKE, FAKE, FAKE, 2, 8, FAKE, FAKE, FAKE, 1 << 20, None]


@pytest.mark.parametrize("fn,args,at,value,status", [
    ("moe_route", ROUTE, 1, 2, -1), ("moe_route", ROUTE, 3, 0, -1), ("moe_route", ROUTE, 3, 4097, -1),
    ("moe_route", ROUTE, 4, 9, -1), ("moe_route", ROUTE, 4, 0, -1), ("moe_route", ROUTE, 2, -1, -1),
    ("moe_route", ROUTE, 6, 2, -1), ("moe_route", ROUTE, 0, None, -1), ("moe_route", ROUTE, 9, None, -1),
    ("moe_route", ROUTE, 0, FAKE + 2, -3), ("moe_route", ROUTE, 5, FAKE + 1, -3), ("moe_route", ROUTE, 2, 1 << 24, -1),
    ("moe_route_bwd", ROUTE_BWD, 5, None, -1), ("moe_route_bwd", ROUTE_BWD, 10, None, -1),
    ("moe_route_bwd", ROUTE_BWD, 10, FAKE + 2, -3), ("moe_route_bwd", ROUTE_BWD, 4, 17, -1),
    ("moe_plan", PLAN, 1, -1, -1), ("moe_plan", PLAN, 1, (1 << 24) + 1, -1), ("moe_plan", PLAN, 2, 0, -1),
    ("moe_plan", PLAN, 2, 4097, -1), ("moe_plan", PLAN, 3, 100, -1), ("moe_plan", PLAN, 3, -128, -1),
    ("moe_plan", PLAN, 0, None, -1), ("moe_plan", PLAN, 8, None, -1), ("moe_plan", PLAN, 9, None, -1),
    ("moe_plan", PLAN, 10, 100, -1), ("moe_plan", PLAN, 9, FAKE + 2, -3), ("moe_plan", PLAN, 7, FAKE + 2, -3),
    ("moe_dispatch", DISPATCH, 2, 24, -1), ("moe_dispatch", DISPATCH, 2, 0, -1), ("moe_dispatch", DISPATCH, 3, 17, -1),
    ("moe_dispatch", DISPATCH, 8, 100, -1), ("moe_dispatch", DISPATCH, 10, FAKE, -1), ("moe_dispatch", DISPATCH, 13, FAKE, -1),
    ("moe_dispatch", DISPATCH, 0, FAKE + 8, -3), ("moe_dispatch", DISPATCH, 12, FAKE + 8, -3), ("moe_dispatch", DISPATCH, 6, None, -1),
    ("moe_dispatch", DISPATCH, 11, 5, -1), ("moe_dispatch", DISPATCH, 7, 0, -1),
    ("moe_combine", COMBINE, 1, 3, -1), ("moe_combine", COMBINE, 4, 8, -1), ("moe_combine", COMBINE, 5, 0, -1),
    ("moe_combine", COMBINE, 0, None, -1), ("moe_combine", COMBINE, 8, FAKE + 2, -3), ("moe_combine", COMBINE, 3, -1, -1),
    ("moe_token_glu", TOKEN_GLU, 2, 48, -1), ("moe_token_glu", TOKEN_GLU, 8, 24, -1), ("moe_token_glu", TOKEN_GLU, 10, 2, -1),
    ("moe_token_glu", TOKEN_GLU, 1, 513, -1), ("moe_token_glu", TOKEN_GLU, 4, None, -1), ("moe_token_glu", TOKEN_GLU, 5, FAKE + 8, -3),
    ("moe_token_linear", TOKEN_LIN, 1, 1025, -1), ("moe_token_linear", TOKEN_LIN, 7, 8, -1), ("moe_token_linear", TOKEN_LIN, 9, None, -1),
    ("moe_token_linear", TOKEN_LIN, 9, FAKE + 4, -3), ("moe_token_linear", TOKEN_LIN, 8, 0, -1),
    ("lora_linear", LORA, 2, 40, -1), ("lora_linear", LORA, 6, 20, -1), ("lora_linear", LORA, 11, 12, -1),
    ("lora_linear", LORA, 11, 136, -1), ("lora_linear", LORA, 10, -1, -1), ("lora_linear", LORA, 7, None, -1),
    ("lora_linear", LORA, 14, None, -1), ("lora_linear", LORA, 15, 16, -1), ("lora_linear", LORA, 13, FAKE + 8, -3),
    ("lora_linear", LORA, 12, FAKE + 2, -3), ("lora_linear", LORA, 1, -1, -1),
])
def test_c_entry_points_refuse(lib, fn, args, at, value, status):
    assert getattr(lib, fn)(*with_change(args, at, value)) == status


def test_glu_entry_points_refuse(lib):
    sp = (ctypes.c_int64 * 2)(128, 128)
    ops = [FAKE] * 6
    for fn, tail in (("moe_glu", lambda s, act: [s, act, FAKE, None, None]),
                     ("moe_glu_bwd", lambda s, act: [s, FAKE, act, FAKE, None])):
        f = getattr(lib, fn)
        assert f(*ops, 256, 24, 128, 2, *tail(sp, 0)) == -1              # f not a multiple of 16
        assert f(*ops, 256, 32, 96, 2, *tail(sp, 0)) == -1               # k not a multiple of 128
        assert f(*ops, 256, 32, 128, 2, *tail(sp, 2)) == -1              # unknown activation
        assert f(*ops, 256, (1 << 19) + 16, 128, 2, *tail(sp, 0)) == -1  # too many lines
        assert f(*ops, 228, 32, 128, 2, *tail((ctypes.c_int64 * 2)(128, 100), 0)) == -2
        assert f(FAKE + 8, *ops[1:], 256, 32, 128, 2, *tail(sp, 0)) == -3
        assert f(None, *ops[1:], 256, 32, 128, 2, *tail(sp, 0)) == -1
        assert f(*ops, 256, 32, 128, 0, *tail(sp, 0)) == -1
    assert lib.moe_glu(*ops, 256, 32, 128, 2, sp, 0, None, None, None) == -1          # no output
    assert lib.moe_glu(*ops, 256, 32, 128, 2, sp, 0, FAKE, FAKE + 8, None) == -3
    assert lib.moe_glu_bwd(*ops, 256, 32, 128, 2, sp, None, 0, FAKE, None) == -1      # no gate values
    assert lib.moe_glu_graphsafe(*ops, 256, 32, 128, 2, None, 0, FAKE, None, FAKE, None) == -1
    assert lib.moe_glu_graphsafe(*ops, 200, 32, 128, 2, FAKE, 0, FAKE, None, FAKE, None) == -1
    assert lib.moe_glu_bwd_graphsafe(*ops, 256, 32, 128, 2, FAKE, FAKE, 0, FAKE, None, None) == -1


def test_nothing_to_do_is_no_error(lib):
    assert lib.moe_route(*with_change(ROUTE, 2, 0)) == 0
    assert lib.moe_combine(*with_change(COMBINE, 3, 0)) == 0
    assert lib.moe_token_linear(*with_change(TOKEN_LIN, 1, 0)) == 0
    assert lib.lora_linear(*with_change(LORA, 1, 0)) == 0


def test_workspace_sizes(lib):
    assert moe.moe_plan_workspace(4096, 512) == 0 and moe.moe_plan_workspace(4097, 512) > 0
    assert moe.moe_plan_workspace(100, 513) > 0
    assert moe.moe_plan_workspace(0, 4096) > 0
    assert moe.lora_workspace(0, 64, 16, 8) == 0
    assert moe.lora_workspace(65, 64, 16, 8) >= 65 * 16 * 4


class _NoCalls:
    def __getattr__(self, name):
        def fail(*args, **kwargs):
            raise AssertionError(f"{name} was called although an argument check should have failed")
        return fail


@pytest.fixture
def cpu_device(monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: torch.device("cpu"))
    monkeypatch.setattr(moe, "_device_index", lambda: -2)  # every buffer through the full checks
    monkeypatch.setattr(moe, "load_library", lambda *a, **k: _NoCalls())
    monkeypatch.setattr(moe, "_stream", lambda *a: None)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


BAD_CALLS = {
    "logits type": (lambda: moe.moe_route(f32(4, 8).double(), i32(4, 2), f32(4, 2)), "logits"),
    "logits order": (lambda: moe.moe_route(f32(8, 4).t(), i32(4, 2), f32(4, 2)), "logits"),
    "ids type": (lambda: moe.moe_route(f32(4, 8), i32(4, 2).long(), f32(4, 2)), "ids"),
    "weights shape": (lambda: moe.moe_route(f32(4, 8), i32(4, 2), f32(4, 3)), "weights"),
    "bias size": (lambda: moe.moe_route(f32(4, 8), i32(4, 2), f32(4, 2), select_bias=f32(7)), "select_bias"),
    "bias device": (lambda: moe.moe_route(f32(4, 8), i32(4, 2), f32(4, 2), select_bias=torch.zeros(8, device="meta")),
                    "select_bias"),
    "dlogits type": (lambda: moe.moe_route_bwd(f32(4, 8), i32(4, 2), f32(4, 2), b16(4, 8)), "dlogits"),
    "rows shape": (lambda: moe.moe_plan(i32(4, 2), i32(8), i32(8), i32(7), i32(128), i32(1)), "rows"),
    "counts size": (lambda: moe.moe_plan(i32(4, 2), i32(8), i32(7), i32(4, 2), i32(128), i32(1)), "counts"),
    "workspace type": (lambda: moe.moe_plan(i32(4, 2), i32(8), i32(8), i32(4, 2), i32(128), i32(1), f32(64)), "workspace"),
    "x type": (lambda: moe.moe_dispatch(f32(4, 64), i32(4, 2), i32(128), i32(8), b16(128, 64)), "x"),
    "out width": (lambda: moe.moe_dispatch(b16(4, 64), i32(4, 2), i32(128), i32(8), b16(128, 32)), "out"),
    "src size": (lambda: moe.moe_dispatch(b16(4, 64), i32(4, 2), i32(127), i32(8), b16(128, 64)), "src"),
    "y alone": (lambda: moe.moe_dispatch(b16(4, 64), i32(4, 2), i32(128), i32(8), b16(128, 64), y=f32(128, 64)), "dweights"),
    "combine rows": (lambda: moe.moe_combine(f32(128, 64), i32(8), b16(4, 64)), "rows"),
    "combine out": (lambda: moe.moe_combine(f32(128, 64), i32(4, 2), b16(4, 32)), "out"),
    "combine y type": (lambda: moe.moe_combine(f32(128, 64).double(), i32(4, 2), b16(4, 64)), "y"),
    "glu lines": (lambda: moe.moe_glu(u8(128, 64), u8(128, 8), f32(128), u8(1, 33, 64), u8(1, 33, 8), f32(33), [128], b16(128, 16)),
                  "up lines"),
    "glu columns": (lambda: moe.moe_glu(u8(128, 64), u8(128, 8), f32(128), u8(1, 32, 32), u8(1, 32, 4), f32(32), [128], b16(128, 16)),
                    "columns"),
    "glu splits": (lambda: moe.moe_glu(u8(128, 64), u8(128, 8), f32(128), u8(1, 32, 64), u8(1, 32, 8), f32(32), [128, 0], b16(128, 16)),
                   "splits"),
    "glu out": (lambda: moe.moe_glu(u8(128, 64), u8(128, 8), f32(128), u8(1, 32, 64), u8(1, 32, 8), f32(32), [128], b16(128, 15)), "h"),
    "glu gu": (lambda: moe.moe_glu_bwd(u8(128, 64), u8(128, 8), f32(128), u8(1, 16, 64), u8(1, 16, 8), f32(16), [128], b16(128, 16),
                                       b16(128, 32)), "gu"),
    "token ids": (lambda: moe.moe_token_linear(b16(4, 64), i32(3), u8(2, 16, 32), u8(2, 16, 4), f32(32), f32(4, 16)), "ids"),
    "token glu h": (lambda: moe.moe_token_glu(b16(4, 64), i32(4, 2), u8(2, 32, 32), u8(2, 32, 4), f32(64), b16(7, 16)), "h"),
    "lora b": (lambda: moe.lora_linear(b16(4, 64), u8(32, 32), u8(32, 4), f32(32), b16(2, 8, 64), b16(2, 31, 8), i32(4), f32(2),
                                       b16(4, 32), u8(1024)), "lora_b"),
    "lora ids": (lambda: moe.lora_linear(b16(4, 64), u8(32, 32), u8(32, 4), f32(32), b16(2, 8, 64), b16(2, 32, 8), i32(3), f32(2),
                                         b16(4, 32), u8(1024)), "adapter_ids"),
    "lora order": (lambda: moe.lora_linear(b16(64, 4).t(), u8(32, 32), u8(32, 4), f32(32), b16(2, 8, 64), b16(2, 32, 8), i32(4),
                                           f32(2), b16(4, 32), u8(1024)), "x"),
}


@pytest.mark.parametrize("name", sorted(BAD_CALLS))
def test_binding_refuses_wrong_buffers(cpu_device, name):
    call, what = BAD_CALLS[name]
    with pytest.raises(ValueError, match=what):
        call()


def test_capacity_holds_any_choice():
    rng = np.random.default_rng(1)
    for T, k, E in ((1, 1, 1), (5, 2, 8), (100, 8, 64), (1000, 3, 7), (1, 8, 256)):
        cap = moe.moe_capacity(T, k, E)
        assert cap % 128 == 0
        for _ in range(20):
            ids = np.stack([rng.permutation(E)[:min(k, E)] for _ in range(T)])
            assert R.plan(ids, E, 0)[1][-1] <= cap
        # the worst choice: one pair above a multiple of 128 in as many experts as can have it
        n, worst = T * k, 0
        for parts in range(1, min(n, E) + 1):
            worst = max(worst, (parts - 1) * 128 + (n - parts + 1 + 127) // 128 * 128)
        assert worst <= cap


def test_launches_past_the_limit_are_refused(lib):
    """Tiles that a launch cannot hold (2^24 work-groups of 256 threads)."""
    rows, ops = 1 << 24, [FAKE] * 6
    sp = (ctypes.c_int64 * 1)(rows)
    assert lib.moe_glu(*ops, rows, 1 << 14, 128, 1, sp, 0, FAKE, None, None) == -1
    assert lib.moe_glu(*ops, rows, 1 << 19, 128, 1, sp, 0, FAKE, FAKE, None) == -1
    assert lib.moe_glu_graphsafe(*ops, rows, 1 << 14, 128, 1, FAKE, 0, FAKE, None, FAKE, None) == -1
    assert lib.moe_glu_bwd(*ops, rows, 1 << 15, 128, 1, sp, FAKE, 0, FAKE, None) == -1
    assert lib.moe_glu_bwd_graphsafe(*ops, rows, 1 << 15, 128, 1, FAKE, FAKE, 0, FAKE, FAKE, None) == -1
    no_adapters = [FAKE, rows, 64, FAKE, FAKE, FAKE, 1 << 15, None, None, None, 0, 8, None, FAKE, FAKE, 1 << 25, None]
    assert lib.lora_linear(*no_adapters) == -1
    assert lib.lora_linear(*with_change(no_adapters, 6, 1 << 20)) == -1


@pytest.mark.parametrize("k,n", [(32, 16), (2048, 528), (7168, 7168), (4896, 7168), (7168, 256), (4096, 1 << 16)])
def test_lora_workspace_serves_smaller_calls(lib, k, n):
    """It grows with the rows and with the rank, and keeps to its bound."""
    ranks = (0, 8, 16, 24, 64, 128)
    before = dict.fromkeys(ranks, 0)
    for tokens in sorted({*range(1, 300), *range(300, 9000, 61), 16384, 32768, 32769, 1 << 20}):
        last = 0
        for rank in ranks:
            size = moe.lora_workspace(tokens, k, n, rank)
            r16 = (rank + 15) // 16 * 16
            kept = (tokens * r16 * 6 + 255) // 256 * 256 + (tokens * 4 + 255) // 256 * 256
            assert last <= size and before[rank] <= size <= max(32 << 20, kept), (tokens, rank)
            last = before[rank] = size


def test_lora_scales_are_four_byte_aligned(lib):
    """As the scales of every other product; the small workspace stops the call."""
    small = with_change(with_change(LORA, 15, 0), 4, FAKE + 4)
    assert lib.lora_linear(*small) == -1
    assert lib.lora_linear(*with_change(small, 4, FAKE + 2)) == -3
