"""Products in 8-bit integers on the GPU: the cast of rows, the projection, the
experts' products and gated block, and the single-token forms.  Integer sums are
exact and every later step is one rounding, so all but the activation is
compared bit by bit with the plain implementation."""
import numpy as np
import pytest
import torch

import i8_reference as I
import moe_reference as R
from gpu_helpers import CANARY, Guarded, log
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import i8, moe

pytestmark = pytest.mark.gpu

ACTS = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}
TYPES = {"f32": (torch.float32, 4), "bf16": (torch.bfloat16, 2)}


def dev(a):
    return R.to_dev(a)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == CANARY).all())


# ------------------------------------------------------------------- cast

def rows_of(rng, m, k):
    """bf16 rows: normal ones of very different size, zeros, the smallest and the largest values, and no numbers."""
    x = rng.standard_normal((m, k)) * np.exp(3 * rng.standard_normal((m, 1)))
    for r, s in enumerate((0.0, 2.0 ** -110, 2.0 ** -130, 3.0e38)):
        if m > r + 1:
            x[r + 1] = np.clip(rng.standard_normal(k), -1, 1) * s
    if m > 6:
        x[5, rng.integers(k)] = np.inf
        x[6, rng.integers(k)] = np.nan
    x = x.astype(np.float32)
    x[0, 0] = -0.0
    return R.bf16_round(x)[0]


CASTS = [(1, 16), (3, 48), (9, 512), (7, 528), (12, 1040), (5, 2064), (8, 4112), (9, 6160), (9, 7168), (8, 8192), (8, 8208),
         (3, 131056), (300, 256), (513, 1040), (600, 2064),
         (16400, 1040), (4200, 4112), (1100, 16400)]  # codes past the caches


@pytest.mark.parametrize("m,k", CASTS)
def test_cast(m, k):
    log(f"cast m={m} k={k}")
    x = rows_of(np.random.default_rng(m * k), m, k)
    q, s = Guarded(m * k, torch.int8, (m, k)), Guarded(4 * m, torch.float32)
    i8.i8_group_cast(x.to("cuda:0"), q.t, s.t)
    torch.cuda.synchronize()
    assert q.guards_intact() and s.guards_intact()
    want_q, want_s = I.cast(x.float().numpy())
    I.same_bits(s.t, want_s, "scale")
    assert np.array_equal(q.numpy(), want_q)
    # what a code stands for is within half a step (and the roundings of quotient, product and scale)
    fin = np.isfinite(want_s)
    step = want_s[fin, None].astype(np.float64)
    off = np.abs(want_q[fin] * step - x.double().numpy()[fin])
    assert (off <= step * (0.5 + 127 * 4 * R.U) + 127 * 2.0 ** -149).all()


def test_cast_device_routing_leaves_the_other_rows():
    for m, spare, k in ((256, 128, 272), (128, 384, 8208)):
        x = rows_of(np.random.default_rng(k), m + spare, k)
        x[m:] = float("nan")
        offs = torch.tensor([128, 128, m], dtype=torch.int32, device="cuda:0")
        status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
        q, s = Guarded((m + spare) * k, torch.int8, (m + spare, k)), Guarded(4 * (m + spare), torch.float32)
        i8.i8_group_cast_graphsafe(x.to("cuda:0"), offs, q.t, s.t, status)
        torch.cuda.synchronize()
        want_q, want_s = I.cast(x.float().numpy()[:m])
        assert int(status) == 0 and q.guards_intact() and s.guards_intact()
        assert np.array_equal(q.numpy()[:m], want_q) and untouched(q.t[m:]) and untouched(s.t[m:])
        I.same_bits(s.t[:m], want_s, "scale")
        for bad, bit in (([100, 128, m], B.NVFP4G_DEV_UNALIGNED), ([256, 128, m], B.NVFP4G_DEV_NONMONO),
                         ([128, 128, m + spare + 128], B.NVFP4G_DEV_OVERFLOW)):
            status.zero_()
            q = Guarded((m + spare) * k, torch.int8, (m + spare, k))
            i8.i8_group_cast_graphsafe(x.to("cuda:0"), torch.tensor(bad, dtype=torch.int32, device="cuda:0"), q.t, s.t, status)
            torch.cuda.synchronize()
            assert int(status) & bit and untouched(q.t)


# ------------------------------------------------------------- projection

def operands(rng, m, n, k, E=None):
    qa, qb = I.random_codes(rng, m, k), I.random_codes(rng, *((n, k) if E is None else (E, n, k)))
    sa = (np.exp(rng.standard_normal(m)) * 1e-2).astype(np.float32)
    sb = (np.exp(rng.standard_normal(qb.shape[:-1])) * 1e-2).astype(np.float32)
    if m > 2:
        sa[1], sa[2] = np.nan, 0.0                                  # a row that was no number, a row of zeros
    return qa, sa, qb, sb


def linear(qa, sa, qb, sb, kind):
    (m, k), n = qa.shape, qb.shape[0]
    t, size = TYPES[kind]
    out = Guarded(size * m * n, t, (m, n))
    ws = torch.full((i8.i8_linear_workspace(m, k, n),), 0xFF, dtype=torch.uint8, device="cuda:0")
    i8.i8_linear(dev(qa), dev(sa), dev(qb), dev(sb), out.t, ws)
    torch.cuda.synchronize()
    assert out.guards_intact()
    return out.t


LINEAR = [  # rows, n, k
    (1, 16, 16), (1, 512, 7168), (3, 48, 128), (5, 272, 80), (16, 1040, 144), (17, 64, 528), (31, 32, 2048), (33, 528, 272),
    (64, 80, 4112), (65, 16, 16), (100, 1024, 1040), (127, 144, 112), (128, 256, 256), (129, 272, 384), (193, 528, 1488),
    (255, 48, 2064), (300, 784, 96), (513, 1040, 208), (1000, 96, 4096), (1030, 2064, 144), (2049, 512, 272),
    (8, 7168, 256), (12, 4096, 13072), (2100, 4112, 144), (9000, 4112, 48), (1500, 2304, 1040), (20, 7168, 1296), (40, 16, 7168),
    (29, 272, 6160), (48, 144, 4112), (63, 4112, 1040), (18, 8208, 2064), (50, 528, 2064), (9, 48, 23056), (16, 8208, 1040), (15, 96, 13328),
    (8, 66064, 272), (20, 66064, 1040), (40, 66064, 1040),  # more work-groups than CUs
]


@pytest.mark.parametrize("m,n,k", LINEAR)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_linear(m, n, k, kind):
    log(f"linear m={m} n={n} k={k} {kind}")
    ops = operands(np.random.default_rng(m + n + k), m, n, k)
    I.same_bits(linear(*ops, kind), I.product(*ops), "out")


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_linear_longest_sums(m):
    """All codes -128 at the largest k: the sum is 2147221504, just below 2^31."""
    n, k = 32, i8.MAX_K
    qa, qb = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    qb[1::2] = 127
    one = lambda c: np.ones(c, np.float32)  # noqa: E731
    I.same_bits(linear(qa, one(m), qb, one(n), "f32"), I.product(qa, one(m), qb, one(n)), "out")


def test_linear_offsets_past_32_bits():
    """Rows of the codes and of the output beyond 4 GiB."""
    n, k, m = 4096, 16384, (1 << 32) // 16384 + 200
    rng = np.random.default_rng(3)
    rows = [0, 1, m - 130, m - 1]
    qa, sa, qb, sb = operands(rng, len(rows), n, k)
    a = torch.zeros((m, k), dtype=torch.int8, device="cuda:0")
    s = torch.zeros(m, device="cuda:0")
    a[rows], s[rows] = dev(qa), dev(sa)
    out = torch.empty((m, n), device="cuda:0")
    ws = torch.empty(i8.i8_linear_workspace(m, k, n), dtype=torch.uint8, device="cuda:0")
    i8.i8_linear(a, s, dev(qb), dev(sb), out, ws)
    I.same_bits(out[rows], I.product(qa, sa, qb, sb), "out")
    rest = torch.ones(m, dtype=torch.bool, device="cuda:0")
    rest[rows] = False
    assert int((out != 0).any(1)[rest].sum()) == 0


# ------------------------------------------------------- experts' products

GROUPS = [  # splits, n, k
    ([128], 16, 16), ([128, 0, 256], 48, 144), ([0, 128], 272, 400), ([256, 128, 0, 0, 128], 144, 640), ([384], 528, 128),
    ([128] * 9, 32, 112), ([0, 0, 640, 128, 0], 1040, 272), ([1024, 0, 1664, 128, 384], 656, 208),
    ([4096, 0, 128, 4224, 256], 528, 144), ([128] * 70 + [0, 384], 272, 80), ([1408, 0, 640, 256, 1152], 4112, 80),
    ([2048, 384, 0, 1664, 4096], 2064, 48), ([640, 0, 384], 1040, 1040), ([8192, 128, 0, 7936, 128], 2064, 400),
]


@pytest.mark.parametrize("splits,n,k", GROUPS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_group_gemm(splits, n, k, kind):
    log(f"group_gemm {splits[:5]} n={n} k={k} {kind}")
    M, E = sum(splits), len(splits)
    ops = operands(np.random.default_rng(n + k), M, n, k, E)
    t, size = TYPES[kind]
    out = Guarded(size * M * n, t, (M, n))
    i8.i8_group_gemm(*[dev(v) for v in ops], splits, out.t)
    torch.cuda.synchronize()
    assert out.guards_intact()
    I.same_bits(out.t, I.grouped(*ops, splits), "out")


def glu_expect(ops, splits, f, kind):
    gu = I.grouped(*ops, splits).astype(np.float64)
    g, u = gu[:, :f], gu[:, f:]
    # g and u are the kernel's own fp32 values: only the activation and two products round
    return R.act(g, kind)[0] * u, R.glu_bound(g, u, 2 * R.U * np.abs(g), 2 * R.U * np.abs(u), kind)


@pytest.mark.parametrize("splits,n,k", GROUPS)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_group_glu(splits, n, k, kind):
    f, M, E = n, sum(splits), len(splits)
    log(f"group_glu {splits[:5]} f={f} k={k} {kind}")
    qa, sa, qb, sb = operands(np.random.default_rng(n + k + 1), M, 2 * f, k, E)
    sa[1] = 0.5                                                     # finite throughout: no row of NaN here
    ops = (qa, sa, qb, (sb * 0.05).astype(np.float32))
    h = Guarded(2 * M * f, torch.bfloat16, (M, f))
    i8.i8_group_glu(*[dev(v) for v in ops], splits, h.t, act=ACTS[kind])
    torch.cuda.synchronize()
    assert h.guards_intact()
    R.check(h.t, *glu_expect(ops, splits, f, kind), "h")


@pytest.mark.parametrize("splits,spare", [([128, 0, 256], 256), ([1024, 0, 1664, 128, 384], 640), ([0, 0], 128)])
@pytest.mark.parametrize("op", ["gemm", "glu"])
def test_device_routing_writes_the_routed_rows_alone(splits, spare, op):
    n, k, M, E = 96, 208, sum(splits), len(splits)
    cap = M + spare
    qa, sa, qb, sb = [dev(v) for v in operands(np.random.default_rng(5), cap, n, k, E)]
    t = torch.bfloat16 if op == "glu" else torch.float32
    width = n // 2 if op == "glu" else n

    def call(offs):
        status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
        out = Guarded(cap * width * t.itemsize, t, (cap, width))
        f = i8.i8_group_glu_graphsafe if op == "glu" else i8.i8_group_gemm_graphsafe
        f(qa, sa, qb, sb, torch.tensor(offs, dtype=torch.int32, device="cuda:0"), out.t, status)
        torch.cuda.synchronize()
        assert out.guards_intact()
        return out.t, int(status)

    out, status = call(B.offsets_from_splits(splits))
    want = torch.empty((M, width), dtype=t, device="cuda:0")
    f = i8.i8_group_glu if op == "glu" else i8.i8_group_gemm
    f(qa[:M].contiguous(), sa[:M].contiguous(), qb, sb, splits, want)
    raw = torch.int16 if op == "glu" else torch.int32
    assert status == 0 and torch.equal(out[:M].view(raw), want.view(raw)) and untouched(out[M:])
    ends = B.offsets_from_splits(splits)
    for bad, bit in ((ends[:-1] + [ends[-1] + 4], B.NVFP4G_DEV_UNALIGNED), ([ends[-1] + 128] + ends[1:], B.NVFP4G_DEV_NONMONO),
                     (ends[:-1] + [cap + 128], B.NVFP4G_DEV_OVERFLOW)):
        out, status = call(bad)
        assert status & bit and untouched(out)


@pytest.mark.parametrize("splits,spare", [([4096, 0, 128, 4224, 256], 128), ([384] * 23 + [0], 1280)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "silu", "gelu"])
def test_device_routing_of_large_tiles(splits, spare, kind):
    """Rows enough for tiles that hold two 128-row groups of an expert, the last of them half empty."""
    glu = kind in ACTS
    n, k, M, E = 2080 if glu else 2064, 400, sum(splits), len(splits)
    cap = M + spare
    rng = np.random.default_rng(M)
    width = n // 2 if glu else n
    qa, qb = (torch.randint(-128, 128, s, dtype=torch.int8, device="cuda:0") for s in ((cap, k), (E, n, k)))
    sa, sb = dev(np.exp(rng.standard_normal(cap)).astype(np.float32)), dev((np.exp(rng.standard_normal((E, n))) * 1e-5).astype(np.float32))
    t, size = (torch.bfloat16, 2) if glu else TYPES[kind]
    out, status = Guarded(size * cap * width, t, (cap, width)), torch.zeros(1, dtype=torch.int32, device="cuda:0")
    offs = torch.tensor(B.offsets_from_splits(splits), dtype=torch.int32, device="cuda:0")
    if glu:
        i8.i8_group_glu_graphsafe(qa, sa, qb, sb, offs, out.t, status, act=ACTS[kind])
    else:
        i8.i8_group_gemm_graphsafe(qa, sa, qb, sb, offs, out.t, status)
    torch.cuda.synchronize()
    assert int(status) == 0 and out.guards_intact() and untouched(out.t[M:])
    rows = np.sort(rng.choice(M, 200, replace=False))
    ends = np.cumsum(splits)
    ops = [v.cpu().numpy() for v in (qa, sa, qb, sb)]
    for r in rows:
        e = int(np.searchsorted(ends, r, side="right"))
        y = I.product(ops[0][r:r + 1], ops[1][r:r + 1], ops[2][e], ops[3][e])
        if glu:
            g, u = y[:, :width].astype(np.float64), y[:, width:].astype(np.float64)
            R.check(out.t[r:r + 1], R.act(g, kind)[0] * u, R.glu_bound(g, u, 2 * R.U * np.abs(g), 2 * R.U * np.abs(u), kind), "h")
        else:
            I.same_bits(out.t[r:r + 1], y, f"row {r}")


def test_no_rows():
    e = lambda *s, t=torch.int8: torch.empty(s, dtype=t, device="cuda:0")  # noqa: E731
    f32 = torch.float32
    i8.i8_group_cast(e(0, 64, t=torch.bfloat16), e(0, 64), e(0, t=f32))
    i8.i8_linear(e(0, 64), e(0, t=f32), e(32, 64), e(32, t=f32), e(0, 32, t=f32))
    i8.i8_group_gemm(e(0, 64), e(0, t=f32), e(2, 32, 64), e(2, 32, t=f32), [0, 0], e(0, 32, t=f32))
    i8.i8_group_glu(e(0, 64), e(0, t=f32), e(2, 32, 64), e(2, 32, t=f32), [0, 0], e(0, 16, t=torch.bfloat16))
    i8.i8_token_linear(e(0, 64, t=torch.bfloat16), e(0, t=torch.int32), e(2, 32, 64), e(2, 32, t=f32), e(0, 32, t=f32))


# ------------------------------------------------------------ single tokens

TOKENS = [  # T, E, topk, k, f
    (1, 1, 1, 16, 16), (1, 8, 8, 176, 48), (3, 4, 2, 112, 16), (17, 4, 2, 128, 64), (33, 1, 1, 272, 32), (64, 8, 8, 256, 80),
    (24, 64, 6, 2048, 128), (2, 3, 3, 7168, 32), (4, 2, 1, 4112, 48), (7, 2, 2, 528, 16), (100, 2, 2, 64, 16), (60, 1, 16, 64, 16),
    (24, 2, 1, 2064, 32), (29, 1, 1, 7168, 32), (32, 16, 8, 96, 1040), (64, 1, 1, 13072, 16), (1, 2, 1, 131056, 16),
    (9, 1, 1, 20000, 32), (16, 64, 4, 272, 1040), (64, 64, 16, 272, 1040), (64, 32, 16, 272, 2064),
]


def token_ids(rng, T, E, topk):
    ids = rng.integers(0, E, (T, topk)).astype(np.int32)       # repeated experts of a token are allowed
    if T > 2:
        ids[1] = -1
        ids[2, 0] = E                                          # out of range: no expert
    return ids


def token_product(xt, ids, qb, sb, topk):
    q, s = I.cast(xt.float().numpy())
    out = np.zeros((ids.size, qb.shape[1]), np.float32)
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < qb.shape[0]:
            out[p] = I.product(q[p // topk:p // topk + 1], s[p // topk:p // topk + 1], qb[e], sb[e])
    return out


@pytest.mark.parametrize("T,E,topk,k,f", TOKENS)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_token_glu(T, E, topk, k, f, kind):
    log(f"token_glu T={T} E={E} topk={topk} k={k} f={f} {kind}")
    rng = np.random.default_rng(T + k)
    qb = I.random_codes(rng, E, 2 * f, k)
    sb = (np.exp(rng.standard_normal((E, 2 * f))) * 0.05 / k ** 0.5).astype(np.float32)
    xt = R.bf16_round(rng.standard_normal((T, k)))[0]
    ids = token_ids(rng, T, E, topk)
    h = Guarded(2 * T * topk * f, torch.bfloat16, (T * topk, f))
    i8.i8_token_glu(xt.to("cuda:0"), dev(ids), dev(qb), dev(sb), h.t, act=ACTS[kind])
    torch.cuda.synchronize()
    assert h.guards_intact()
    gu = token_product(xt, ids, qb, sb, topk).astype(np.float64)
    g, u = gu[:, :f], gu[:, f:]
    R.check(h.t, R.act(g, kind)[0] * u, R.glu_bound(g, u, 2 * R.U * np.abs(g), 2 * R.U * np.abs(u), kind), "h")


@pytest.mark.parametrize("T,E,topk,k,f", TOKENS)
def test_token_linear(T, E, topk, k, f):
    log(f"token_linear T={T} E={E} topk={topk} k={k} n={f}")
    rng = np.random.default_rng(T + k + 1)
    pairs = T * topk
    _, _, qb, sb = operands(rng, 1, f, k, E)
    ids = token_ids(rng, T, E, topk)
    xt = rows_of(rng, pairs, k)
    out = Guarded(4 * pairs * f, torch.float32, (pairs, f))
    i8.i8_token_linear(xt.to("cuda:0"), dev(ids), dev(qb), dev(sb), out.t)
    torch.cuda.synchronize()
    assert out.guards_intact()
    I.same_bits(out.t, token_product(xt, ids, qb, sb, 1), "out")


@pytest.mark.parametrize("pairs,E,k", [(100, 32, 272), (1024, 300, 528), (128, 8, 1040), (999, 16, 64)])
def test_all_tokens_choose_one_expert_of_many(pairs, E, k):
    """More rows for one expert than its share: further passes over them."""
    log(f"one expert pairs={pairs} E={E} k={k}")
    rng, f = np.random.default_rng(pairs), 48
    xt = R.bf16_round(rng.standard_normal((pairs, k)))[0]
    qb, sb = rng.integers(-128, 128, (E, 2 * f, k), dtype=np.int8), np.full((E, 2 * f), 0.01 / k ** 0.5, np.float32)
    ids = np.full((pairs, 1), E - 2, np.int32)
    ids[pairs // 2] = 0
    y, h = Guarded(4 * pairs * 2 * f, torch.float32, (pairs, 2 * f)), Guarded(2 * pairs * f, torch.bfloat16, (pairs, f))
    i8.i8_token_linear(xt.to("cuda:0"), dev(ids), dev(qb), dev(sb), y.t)
    i8.i8_token_glu(xt.to("cuda:0"), dev(ids), dev(qb), dev(sb), h.t)
    torch.cuda.synchronize()
    assert y.guards_intact() and h.guards_intact()
    q, s = I.cast(xt.float().numpy())
    want = I.product(q, s, qb[E - 2], sb[E - 2])
    want[pairs // 2] = I.product(q[pairs // 2:pairs // 2 + 1], s[pairs // 2:pairs // 2 + 1], qb[0], sb[0])[0]
    I.same_bits(y.t, want, "out")
    g, u = want[:, :f].astype(np.float64), want[:, f:].astype(np.float64)
    R.check(h.t, R.act(g, "silu")[0] * u, R.glu_bound(g, u, 2 * R.U * np.abs(g), 2 * R.U * np.abs(u), "silu"), "h")


def test_token_projection_and_grouped_forms_agree():
    """One definition: the same bits from the single-token form, the projection and the experts' product."""
    rng = np.random.default_rng(8)
    T, k, n = 128, 1040, 272
    xt = R.bf16_round(rng.standard_normal((T, k)))[0].to("cuda:0")
    _, _, qb, sb = operands(rng, 1, n, k, 1)
    qb, sb = dev(qb), dev(sb)
    made = i8.alloc_cast(T, k)
    i8.i8_group_cast(xt, **made)
    y = [torch.empty((T, n), device="cuda:0") for _ in range(3)]
    i8.i8_token_linear(xt, torch.zeros(T, dtype=torch.int32, device="cuda:0"), qb, sb, y[0])
    ws = torch.empty(i8.i8_linear_workspace(T, k, n), dtype=torch.uint8, device="cuda:0")
    i8.i8_linear(*made.values(), qb[0], sb[0], y[1], ws)
    i8.i8_group_gemm(*made.values(), qb, sb, [T], y[2])
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    for rows in (1, 5, 33, 70):
        few = torch.empty((rows, n), device="cuda:0")
        ws = torch.empty(i8.i8_linear_workspace(rows, k, n), dtype=torch.uint8, device="cuda:0")
        i8.i8_linear(made["q"][:rows], made["scale"][:rows], qb[0], sb[0], few, ws)
        assert torch.equal(few, y[0][:rows])


DEVICE = [  # splits, spare rows, n (f of the gated block), k: few tiles, long contractions
    ([128, 0, 256], 128, 528, 1040), ([128, 0, 256], 128, 272, 2064), ([0, 384, 128, 0], 256, 1040, 2064),
    ([256, 0, 0, 128], 128, 48, 1296), ([128] * 7 + [0], 128, 144, 7168), ([0, 0, 128], 0, 16, 4112), ([0, 0], 256, 64, 1040),
]


@pytest.mark.parametrize("splits,spare,n,k", DEVICE)
@pytest.mark.parametrize("kind", ["f32", "bf16", "silu", "gelu"])
def test_device_routing_of_long_contractions(splits, spare, n, k, kind):
    """The tiles with four stages under device routing (test_i8_host.py shows that these cases take them): experts
    without rows, rows past the last group left as they were."""
    log(f"device routing {splits} + {spare} n={n} k={k} {kind}")
    glu, M, E = kind in ACTS, sum(splits), len(splits)
    cap = M + spare
    qa, sa, qb, sb = operands(np.random.default_rng(n + k + 2), cap, 2 * n if glu else n, k, E)
    sb = (sb * np.float32(1e-4)).astype(np.float32)
    if glu:
        sa[1] = 0.5                                                 # finite throughout
    t, size = (torch.bfloat16, 2) if glu else TYPES[kind]
    out, status = Guarded(size * cap * n, t, (cap, n)), torch.zeros(1, dtype=torch.int32, device="cuda:0")
    ops = [dev(v) for v in (qa, sa, qb, sb)]
    f, more = (i8.i8_group_glu_graphsafe, dict(act=ACTS[kind])) if glu else (i8.i8_group_gemm_graphsafe, {})

    def call(offs, out):
        f(*ops, torch.tensor(offs, dtype=torch.int32, device="cuda:0"), out, status, **more)
        torch.cuda.synchronize()

    call(B.offsets_from_splits(splits), out.t)
    assert int(status) == 0 and out.guards_intact() and untouched(out.t[M:])
    if M:
        own = (qa[:M], sa[:M], qb, sb)
        if glu:
            R.check(out.t[:M], *glu_expect(own, splits, n, kind), "h")
        else:
            I.same_bits(out.t[:M], I.grouped(*own, splits), "out")
    out.t.view(torch.uint8).fill_(CANARY)
    call([0] * (E - 1) + [cap + 128], out.t)
    assert int(status) & B.NVFP4G_DEV_OVERFLOW and untouched(out.t) and out.guards_intact()
