"""The experts' gated feed-forward block on the GPU: the grouped NVFP4 form
(forward and backward, host splits and device routing) and the single-token
form, against the plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import moe_reference as R
from gpu_helpers import CANARY, Guarded, log
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import moe

pytestmark = pytest.mark.gpu

ACTS = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}


def factor(amax):
    return amax.astype(np.float64) / 2688.0


def case(seed, splits, f, k, lines):
    rng = np.random.default_rng(seed)
    M, E = sum(splits), len(splits)
    a = R.random_lines(rng, M, k)
    b = R.random_lines(rng, E * lines, k, big=8.0 / k)
    return rng, M, E, a, b


def on_device(a, b, E, lines):
    return [R.to_dev(v) for v in a] + [R.to_dev(b[0].reshape(E, lines, -1)), R.to_dev(b[1].reshape(E, lines, -1)),
                                       R.to_dev(b[2])]


def products(a, b, splits, lines, k):
    xa, xb = R.decode(*a[:2]), R.decode(*b[:2])
    fa, fb = factor(a[2]), factor(b[2])
    out, mag, at = [], [], 0
    for e, m in enumerate(splits):
        s = slice(e * lines, (e + 1) * lines)
        p, q = R.product(xa[at:at + m], fa[at:at + m], xb[s], fb[s])
        out.append(p)
        mag.append(R.gemm_bound(q, k))
        at += m
    return np.concatenate(out), np.concatenate(mag)


CASES = [([128], 16, 128), ([128, 0, 256], 48, 384), ([0, 128], 128, 256), ([256, 128, 0, 0, 128], 144, 640),
         ([384], 272, 128), ([128] * 9, 32, 128)]


@pytest.mark.parametrize("splits,f,k", CASES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward(splits, f, k, kind):
    log(f"glu {splits} f={f} k={k} {kind}")
    rng, M, E, a, b = case(f + k, splits, f, k, 2 * f)
    dev = on_device(a, b, E, 2 * f)
    gu, err = products(a, b, splits, 2 * f, k)
    g, u, dg, du = gu[:, :f], gu[:, f:], err[:, :f], err[:, f:]
    want = R.act(g, kind)[0] * u
    for keep in (True, False):
        h = Guarded(2 * M * f, torch.bfloat16, (M, f))
        kept = Guarded(4 * M * f, torch.bfloat16, (M, 2 * f)) if keep else None
        moe.moe_glu(*dev, splits, h.t, gu=kept.t if keep else None, act=ACTS[kind])
        torch.cuda.synchronize()
        assert h.guards_intact()
        R.check(h.t, want, R.glu_bound(g, u, dg, du, kind), "h")
        if keep:
            assert kept.guards_intact()
            R.check(kept.t, gu, err + R.UB * (np.abs(gu) + err), "gu")


@pytest.mark.parametrize("splits,f,k", CASES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward(splits, f, k, kind):
    log(f"glu_bwd {splits} f={f} k={k} {kind}")
    rng, M, E, a, b = case(f + k + 1, splits, f, k, f)
    dev = on_device(a, b, E, f)
    gut, gu = R.bf16_round(rng.standard_normal((M, 2 * f)) * 3)
    if M:
        gut[0, :] = gut[0, :] * 1e4          # a saturated gate
        gu = gut.double().numpy()
    dh, err = products(a, b, splits, f, k)
    out = Guarded(4 * M * f, torch.bfloat16, (M, 2 * f))
    moe.moe_glu_bwd(*dev, splits, gut.to("cuda:0"), out.t, act=ACTS[kind])
    torch.cuda.synchronize()
    assert out.guards_intact()
    g, u = gu[:, :f], gu[:, f:]
    with np.errstate(over="ignore"):
        v, d = R.act(g, kind)
        rel = R.act_rel(g, kind)
    want = np.concatenate([dh * u * d, dh * v], 1)
    # act'(g) = q + g q (1 - q) v': q's relative error, and that of 1 - q, which is absolute in q
    slope = rel * (np.abs(d) + 1) + np.abs(v) * 8 * R.U * (1 + g ** 2)
    eg = err * np.abs(u) * (np.abs(d) + slope) + np.abs(dh * u) * (slope + 8 * R.U)
    eu = err * np.abs(v) * (1 + rel) + np.abs(dh * v) * (rel + 8 * R.U)
    e = np.concatenate([eg, eu], 1) + 1e-30
    R.check(out.t, want, e + R.UB * (np.abs(want) + e), "dgu")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_follows_differences(kind):
    """dh is exact here (one contraction step of small integers), and the
    loss sum(dh * act(g) * u) is differenced in 64 bits at the gu in hand."""
    rng = np.random.default_rng(2)
    f, k, M = 16, 128, 128
    a = (np.full((M, k // 2), 0x22, np.uint8), np.full((M, k // 16), 0x38, np.uint8), np.full(M, 2688, np.float32))
    b = (rng.integers(0, 3, (f, k // 2), dtype=np.uint8) * 2, np.full((f, k // 16), 0x38, np.uint8), np.full(f, 2688, np.float32))
    gut, gu = R.bf16_round(rng.standard_normal((M, 2 * f)))
    out = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_bwd(*on_device(a, b, 1, f), [M], gut.to("cuda:0"), out, act=ACTS[kind])
    dh, _ = R.product(R.decode(*a[:2]), factor(a[2]), R.decode(*b[:2]), factor(b[2]))
    eps = 1e-5

    def loss(x):
        return dh * R.act(x[:, :f], kind)[0] * x[:, f:]

    num = np.empty((M, 2 * f))
    for c in range(2):
        d = np.zeros((M, 2 * f))
        d[:, c * f:(c + 1) * f] = eps
        num[:, c * f:(c + 1) * f] = (loss(gu + d) - loss(gu - d)) / (2 * eps)
    # bf16's rounding, fp32 inside, and eps^2 of the difference on values up to |dh u|
    R.check(out, num, R.UB * np.abs(num) * 1.01 + 1e-5 * (1 + np.abs(dh).max()) * (1 + np.abs(gu).max()), "dgu")


@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_device_routing_writes_the_routed_rows_alone(direction):
    splits, f, k, spare = [128, 0, 256], 48, 256, 256
    lines = 2 * f if direction == "forward" else f
    rng, M, E, a, b = case(11, splits, f, k, lines)
    cap = M + spare
    pad = [np.concatenate([v, np.full((spare, *v.shape[1:]), 0x7F, v.dtype)]) for v in a]
    dev = on_device(pad, b, E, lines)
    exact = on_device(a, b, E, lines)
    offs = torch.tensor(B.offsets_from_splits(splits), dtype=torch.int32, device="cuda:0")
    gu = R.bf16_round(rng.standard_normal((cap, 2 * f)))[0].to("cuda:0")

    def call(o, width):
        status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
        out = Guarded(2 * cap * width, torch.bfloat16, (cap, width))
        if direction == "forward":
            moe.moe_glu_graphsafe(*dev, o, out.t, status)
        else:
            moe.moe_glu_bwd_graphsafe(*dev, o, gu, out.t, status)
        torch.cuda.synchronize()
        assert out.guards_intact()
        return out, int(status)

    width = f if direction == "forward" else 2 * f
    out, status = call(offs, width)
    want = torch.empty((M, width), dtype=torch.bfloat16, device="cuda:0")
    if direction == "forward":
        moe.moe_glu(*exact, splits, want)
    else:
        moe.moe_glu_bwd(*exact, splits, gu[:M].contiguous(), want)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(out.t[:M], want)
    assert (out.t[M:].contiguous().view(torch.uint8).cpu().numpy() == CANARY).all()
    for bad, bit in (([100, 128, 384], B.NVFP4G_DEV_UNALIGNED), ([256, 128, 384], B.NVFP4G_DEV_NONMONO),
                     ([128, 128, cap + 128], B.NVFP4G_DEV_OVERFLOW)):
        out, status = call(torch.tensor(bad, dtype=torch.int32, device="cuda:0"), width)
        assert status & bit
        assert (out.t.view(torch.uint8).cpu().numpy() == CANARY).all()


def test_no_rows():
    f, k = 16, 128
    rng, M, E, a, b = case(1, [128, 0], f, k, 2 * f)
    dev = on_device(a, b, E, 2 * f)
    empty = [t[:0].contiguous() for t in dev[:3]]
    moe.moe_glu(*empty, *dev[3:], [0, 0], torch.empty((0, f), dtype=torch.bfloat16, device="cuda:0"))


# ------------------------------------------------------------ single tokens

TOKENS = [  # T, E, topk, k, f
    (1, 1, 1, 32, 16), (1, 8, 8, 160, 48), (3, 4, 2, 96, 16), (17, 4, 2, 128, 64), (33, 1, 1, 288, 32),
    (64, 8, 8, 256, 80), (24, 64, 6, 2048, 128), (2, 3, 3, 7168, 32), (100, 2, 2, 64, 16), (60, 1, 16, 64, 16),
]


def token_ids(rng, T, E, topk):
    ids = rng.integers(0, E, (T, topk)).astype(np.int32)       # repeated experts of a token are allowed
    if T > 2:
        ids[1] = -1
        ids[2, 0] = E                                          # out of range: no expert
    return ids


def token_products(x, ids, b, E, lines, k):
    xb, fb = R.decode(*b[:2]).reshape(E, lines, k), factor(b[2]).reshape(E, lines)
    out, mag = np.zeros((ids.size, lines)), np.zeros((ids.size, lines))
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            out[p] = (xb[e] @ x[p]) * fb[e]
            mag[p] = (np.abs(xb[e]) @ np.abs(x[p])) * fb[e]
    return out, R.gemm_bound(mag, k)


@pytest.mark.parametrize("T,E,topk,k,f", TOKENS)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_token_glu(T, E, topk, k, f, kind):
    log(f"token_glu T={T} E={E} topk={topk} k={k} f={f} {kind}")
    rng = np.random.default_rng(T + k)
    b = R.random_lines(rng, E * 2 * f, k, big=8.0 / k)
    xt, x = R.bf16_round(rng.standard_normal((T, k)))
    ids = token_ids(rng, T, E, topk)
    h = Guarded(2 * T * topk * f, torch.bfloat16, (T * topk, f))
    moe.moe_token_glu(xt.to("cuda:0"), R.to_dev(ids), R.to_dev(b[0].reshape(E, 2 * f, -1)),
                      R.to_dev(b[1].reshape(E, 2 * f, -1)), R.to_dev(b[2]), h.t, act=ACTS[kind])
    torch.cuda.synchronize()
    assert h.guards_intact()
    gu, err = token_products(np.repeat(x, topk, 0), ids, b, E, 2 * f, k)
    g, u, dg, du = gu[:, :f], gu[:, f:], err[:, :f], err[:, f:]
    R.check(h.t, R.act(g, kind)[0] * u, R.glu_bound(g, u, dg, du, kind), "h")


@pytest.mark.parametrize("T,E,topk,k,f", TOKENS)
def test_token_linear(T, E, topk, k, f):
    log(f"token_linear T={T} E={E} topk={topk} k={k} n={f}")
    rng = np.random.default_rng(T + k + 1)
    b = R.random_lines(rng, E * f, k, big=8.0 / k)
    ids = token_ids(rng, T, E, topk)
    xt, x = R.bf16_round(rng.standard_normal((T * topk, k)) * np.exp(4 * rng.standard_normal((T * topk, 1))))
    out = Guarded(4 * T * topk * f, torch.float32, (T * topk, f))
    args = (R.to_dev(ids), R.to_dev(b[0].reshape(E, f, -1)), R.to_dev(b[1].reshape(E, f, -1)), R.to_dev(b[2]))
    moe.moe_token_linear(xt.to("cuda:0"), *args, out.t)
    torch.cuda.synchronize()
    assert out.guards_intact()
    want, err = token_products(x, ids, b, E, f, k)
    R.check(out.t, want, err, "out")
    assert (out.t.cpu().numpy()[(ids.reshape(-1) < 0) | (ids.reshape(-1) >= E)] == 0).all()
    # a row that overflows stays in its own row
    xt[0] = float("inf")
    again = torch.empty_like(out.t)
    moe.moe_token_linear(xt.to("cuda:0"), *args, again)
    assert torch.equal(again[1:], out.t[1:])


def test_token_and_grouped_forms_agree():
    """Tokens that NVFP4 holds exactly give the same block in both forms, up to
    the order of the sums."""
    rng = np.random.default_rng(8)
    T, k, f = 5, 256, 64
    codes = rng.integers(0, 256, (T, k // 2), dtype=np.uint8)
    a = (codes, np.full((T, k // 16), 0x38, np.uint8), np.full(T, 2688, np.float32))
    b = R.random_lines(rng, 2 * f, k, big=4.0 / k)
    x = torch.from_numpy(R.decode(*a[:2])).to(torch.bfloat16).to("cuda:0")
    rows = [np.concatenate([v, np.zeros((128 - T, *v.shape[1:]), v.dtype)]) for v in a]
    dev = on_device(rows, b, 1, 2 * f)
    h1 = torch.empty((128, f), dtype=torch.bfloat16, device="cuda:0")
    h2 = torch.empty((T, f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu(*dev, [128], h1)
    moe.moe_token_glu(x, torch.zeros((T, 1), dtype=torch.int32, device="cuda:0"), *dev[3:], h2)
    gu, err = products(tuple(rows), b, [128], 2 * f, k)
    bound = 2 * R.glu_bound(gu[:T, :f], gu[:T, f:], err[:T, :f], err[:T, f:], "silu")
    R.check(h2, h1[:T].double().cpu().numpy(), bound, "h")


# ------------------------------------------- wide tiles (more than 128 of them)

# rows, columns, contraction: with 128 (forward) or 256 (backward) columns a
# tile, at least 129 tiles, the last column of them 16 wide; empty experts; one
# case of several scale blocks, one of more than 512 tiles (their XCD order).
WIDE = {"forward": [([1024, 0, 1536, 128, 384], 656, 640), ([16384, 0, 128, 16512], 144, 128)],
        "backward": [([2048, 0, 3072, 128, 384], 528, 640), ([16384, 0, 128, 16512], 272, 128)]}


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_wide_tiles(at, kind):
    splits, f, k = WIDE["forward"][at]
    assert sum(splits) // 128 * -(-f // 128) > 128 * (1 + 3 * at)
    test_forward(splits, f, k, kind)


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_wide_tiles(at, kind):
    splits, f, k = WIDE["backward"][at]
    assert sum(splits) // 128 * -(-f // 256) > 128 * (1 + 3 * at)
    test_backward(splits, f, k, kind)


@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_device_routing_wide_tiles(direction):
    """The host-split call's bits in the routed rows, nothing in the others."""
    splits, f, k = WIDE[direction][0]
    spare = 640
    lines = 2 * f if direction == "forward" else f
    rng, M, E, a, b = case(17, splits, f, k, lines)
    cap = M + spare
    pad = [np.concatenate([v, np.full((spare, *v.shape[1:]), 0x7F, v.dtype)]) for v in a]
    dev, exact = on_device(pad, b, E, lines), on_device(a, b, E, lines)
    offs = torch.tensor(B.offsets_from_splits(splits), dtype=torch.int32, device="cuda:0")
    status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    width = f if direction == "forward" else 2 * f
    out = Guarded(2 * cap * width, torch.bfloat16, (cap, width))
    gu = Guarded(4 * cap * f, torch.bfloat16, (cap, 2 * f))
    want = torch.empty((M, width), dtype=torch.bfloat16, device="cuda:0")
    if direction == "forward":
        want_gu = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
        moe.moe_glu_graphsafe(*dev, offs, out.t, status, gu=gu.t)
        moe.moe_glu(*exact, splits, want, gu=want_gu)
        torch.cuda.synchronize()
        assert gu.guards_intact() and torch.equal(gu.t[:M], want_gu)
        assert (gu.t[M:].contiguous().view(torch.uint8) == CANARY).all()
    else:
        gu.t.copy_(R.bf16_round(rng.standard_normal((cap, 2 * f)))[0])
        moe.moe_glu_bwd_graphsafe(*dev, offs, gu.t, out.t, status)
        moe.moe_glu_bwd(*exact, splits, gu.t[:M].contiguous(), want)
        torch.cuda.synchronize()
    assert int(status) == 0 and out.guards_intact() and torch.equal(out.t[:M], want)
    assert (out.t[M:].contiguous().view(torch.uint8) == CANARY).all()


# --------------------------------------- two token tiles (17 to 32 rows a pass)

TWO_TILES = [(24, 2, 1, 64, 48), (24, 2, 1, 2080, 32), (20, 2, 2, 544, 80), (40, 2, 1, 1056, 16), (29, 1, 1, 7168, 32),
             (32, 16, 8, 96, 1040)]


@pytest.mark.parametrize("T,E,topk,k,f", TWO_TILES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_token_glu_two_tiles(T, E, topk, k, f, kind):
    test_token_glu(T, E, topk, k, f, kind)


@pytest.mark.parametrize("T,E,topk,k,f", TWO_TILES)
def test_token_linear_two_tiles(T, E, topk, k, f):
    test_token_linear(T, E, topk, k, f)
