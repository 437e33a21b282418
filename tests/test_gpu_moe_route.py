"""Selection of experts, its gradient and the plan of the packed groups on
the GPU, against the plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import moe_reference as R
from gpu_helpers import Guarded, log
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import moe

pytestmark = pytest.mark.gpu

SCORES = {"softmax": moe.SCORE_SOFTMAX, "sigmoid": moe.SCORE_SIGMOID}


def logits_for(rng, T, E, kind):
    l = rng.standard_normal((T, E)).astype(np.float32) * 2
    if kind == "ties":           # few distinct values, both zeros among them
        l = np.round(l).astype(np.float32)
        l[l == 0] = rng.choice(np.array([0.0, -0.0], np.float32), (l == 0).sum())
    elif kind == "masks":
        l[rng.random((T, E)) < 0.5] = -np.inf
        l[rng.random((T, E)) < 0.1] = np.nan
        l[rng.random((T, E)) < 0.02] = np.inf
        l[rng.random((T, E)) < 0.1] = -R.FLT_MAX       # the lowest finite value is not a mask
        l[T // 2] = -np.inf                              # a row with nothing left
        if T > 2:
            l[0] = np.nan
    return l


def run_route(l, k, bias, score, normalize, scale, dtype):
    T, E = l.shape
    dev = torch.from_numpy(l).to("cuda:0").to(dtype)
    ids, w = Guarded(4 * T * k, torch.int32, (T, k)), Guarded(4 * T * k, torch.float32, (T, k))
    moe.moe_route(dev, ids.t, w.t, select_bias=None if bias is None else torch.from_numpy(bias).to("cuda:0"),
                  score=SCORES[score], normalize=normalize, scale=scale)
    torch.cuda.synchronize()
    assert ids.guards_intact() and w.guards_intact()
    return dev.float().cpu().numpy(), ids.numpy(), w.numpy()


def weight_tolerance(l, ids, E):
    """Relative: a subtraction and an exponential whose argument is at most
    the spread of the finite logits off its top (that many u), sums of E terms
    (a tree over lanes of at most 64 serial ones), division and scale."""
    c = R.clean(l)
    fin = np.where(np.isfinite(c), c, np.nan)
    with np.errstate(all="ignore"):
        spread = np.nanmax(np.where(np.isnan(fin), 0.0, fin), 1) - np.nanmin(np.where(np.isnan(fin), 0.0, fin), 1)
    return (2 * np.minimum(spread, 200.0) + 96)[:, None] * R.U


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,kind,dtype,biased", [
    (1, 1, 1, "normal", torch.float32, False),
    (5, 7, 7, "ties", torch.float32, True),
    (130, 8, 2, "masks", torch.bfloat16, False),
    (67, 64, 6, "ties", torch.bfloat16, False),
    (33, 100, 10, "normal", torch.bfloat16, True),
    (65, 256, 8, "masks", torch.float32, True),
    (9, 384, 16, "ties", torch.float32, True),
    (6, 513, 16, "masks", torch.bfloat16, False),
    (3, 4096, 16, "normal", torch.float32, False),
    (3, 4095, 5, "ties", torch.bfloat16, True),
])
def test_route(T, E, k, kind, dtype, biased, score, normalize):
    log(f"route T={T} E={E} k={k} {kind} {dtype} {score} {normalize}")
    rng = np.random.default_rng(T * 7 + E)
    bias = rng.standard_normal(E).astype(np.float32).round(1) if biased else None
    l, ids, w = run_route(logits_for(rng, T, E, kind), k, bias, score, normalize, 2.5, dtype)
    want_ids = R.select(l, k, bias)
    assert np.array_equal(ids, want_ids)
    want = R.route_weights(l, want_ids, score, normalize, 2.5)
    # where a chosen score underflows fp32 (below 2^-126) the flush is absolute
    R.check(w, want, weight_tolerance(l, ids, E) * np.abs(want) + 2.5 * 2.0 ** -120, "weights")
    assert (w[ids < 0] == 0).all()


def test_route_without_tokens():
    moe.moe_route(torch.empty((0, 8), device="cuda:0"), torch.empty((0, 2), dtype=torch.int32, device="cuda:0"),
                  torch.empty((0, 2), device="cuda:0"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,kind,dtype", [
    (1, 1, 1, "normal", torch.float32), (5, 7, 3, "ties", torch.float32), (131, 64, 6, "masks", torch.bfloat16),
    (66, 100, 10, "masks", torch.float32), (17, 512, 16, "normal", torch.bfloat16), (3, 4096, 8, "masks", torch.float32),
])
def test_route_gradient_follows_the_formula(T, E, k, kind, dtype, score, normalize):
    log(f"route_bwd T={T} E={E} k={k} {kind} {dtype} {score} {normalize}")
    rng = np.random.default_rng(T + E)
    raw = logits_for(rng, T, E, kind)
    if kind == "masks":
        raw[np.abs(raw) == R.FLT_MAX] = -np.inf     # a finite range for the bound below
        raw[raw == np.inf] = 3.0
    dev = torch.from_numpy(raw).to("cuda:0").to(dtype)
    l = dev.float().cpu().numpy()
    ids = R.select(l, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    size = 4 if dtype == torch.float32 else 2
    out = Guarded(size * T * E, dtype, (T, E))
    moe.moe_route_bwd(dev, R.to_dev(ids), R.to_dev(dw), out.t, score=SCORES[score], normalize=normalize, scale=2.5)
    torch.cuda.synchronize()
    assert out.guards_intact()
    want = R.route_grad(l, ids, dw, score, normalize, 2.5)
    # every term is a weight (bounded as above) times a sum of at most k products of size scale * |dw|
    size_of = 2.5 * np.abs(dw).max(1, keepdims=True)
    bound = (weight_tolerance(l, ids, E) + 4 * k * R.U) * size_of * 2 + 1e-30
    if dtype == torch.bfloat16:
        bound = bound + R.UB * np.abs(want)
    R.check(out.t, want, bound, "dlogits")
    masked = ~(R.clean(l) > -np.inf)
    assert (out.t.float().cpu().numpy()[masked] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_follows_differences(score, normalize):
    rng = np.random.default_rng(3)
    T, E, k, eps = 4, 12, 4, 1e-5
    l = rng.standard_normal((T, E)).astype(np.float32)
    ids = R.select(l, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.empty((T, E), device="cuda:0")
    moe.moe_route_bwd(R.to_dev(l), R.to_dev(ids), R.to_dev(dw), out, score=SCORES[score], normalize=normalize, scale=1.5)
    num = np.zeros((T, E))
    for i in range(E):
        d = np.zeros((T, E))
        d[:, i] = eps
        up = R.route_weights(l.astype(np.float64) + d, ids, score, normalize, 1.5)
        dn = R.route_weights(l.astype(np.float64) - d, ids, score, normalize, 1.5)
        num[:, i] = ((up - dn) * dw).sum(1) / (2 * eps)
    # differences: eps^2 times a third derivative of order one, 1e-16/eps of rounding; the kernel's fp32
    R.check(out, num, 1e-6 * (1 + np.abs(dw).sum(1, keepdims=True)), "dlogits")


PLANS = [(0, 4), (1, 1), (1, 4096), (63, 8), (64, 8), (65, 8), (1000, 3), (4096, 512), (4097, 64), (5000, 513), (3000, 4096),
         (16384, 500), (16385, 40), (40000, 2100), (100003, 256)]


@pytest.mark.parametrize("pairs,E", PLANS)
@pytest.mark.parametrize("spread", ["even", "skewed", "one"])
def test_plan(pairs, E, spread):
    log(f"plan pairs={pairs} E={E} {spread}")
    rng = np.random.default_rng(pairs + E)
    if spread == "even":
        ids = rng.integers(-1, E + 1, pairs)            # invalid ids on both sides
    elif spread == "skewed":
        ids = np.minimum((E * rng.random(pairs) ** 4).astype(np.int64), E - 1)
    else:
        ids = np.full(pairs, E - 1)
    ids = ids.astype(np.int32)
    need = int(R.plan(ids, E, 0)[1][-1])
    for cap in {need, need + 256, max(0, need // 2 // 128 * 128)}:
        g = {n: Guarded(4 * m, torch.int32) for n, m in (("offs", E), ("counts", E), ("rows", pairs), ("src", cap))}
        status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
        ws = torch.full((max(moe.moe_plan_workspace(pairs, E), 1),), 0xA5, dtype=torch.uint8, device="cuda:0")
        moe.moe_plan(R.to_dev(ids), g["offs"].t, g["counts"].t, g["rows"].t, g["src"].t, status, ws)
        torch.cuda.synchronize()
        counts, ends, rows, src = R.plan(ids, E, cap)
        for n, want in (("offs", ends), ("counts", counts), ("rows", rows), ("src", src)):
            assert g[n].guards_intact(), n
            assert np.array_equal(g[n].numpy(), want), n
        assert int(status) == (B.NVFP4G_DEV_OVERFLOW if need > cap else 0)


def test_plan_refuses_a_small_workspace():
    E, pairs = 64, 20000
    i32 = dict(dtype=torch.int32, device="cuda:0")
    args = (torch.zeros(pairs, **i32), torch.zeros(E, **i32), torch.zeros(E, **i32), torch.zeros(pairs, **i32),
            torch.zeros(128, **i32), torch.zeros(1, **i32))
    small = torch.empty(moe.moe_plan_workspace(pairs, E) - 1, dtype=torch.uint8, device="cuda:0")
    for ws in (None, small):
        with pytest.raises(moe.Nvfp4GroupError):
            moe.moe_plan(*args, ws)


def test_route_and_plan_replay_in_a_graph():
    """Captured once, replayed under new logits with eager work between; every
    replay equals the eager calls."""
    rng = np.random.default_rng(9)
    T, E, k = 700, 64, 6
    l = torch.empty((T, E), device="cuda:0")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda:0"), torch.empty((T, k), device="cuda:0")
    p = moe.alloc_plan(T, k, E)

    def step():
        moe.moe_route(l, ids, w)
        moe.moe_plan(ids, **p)

    l.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        l.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (ids, w, p["d_offs"], p["counts"], p["rows"], p["src"])]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (ids, w, p["d_offs"], p["counts"], p["rows"], p["src"])):
            assert torch.equal(a, b)
    assert int(p["d_status"]) == 0


# Up to 8 of 65-128, 257-512 and 513-1024 experts: three more ways to share a
# wave among tokens.
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,kind,dtype,biased", [
    (131, 65, 8, "masks", torch.float32, True), (97, 128, 6, "ties", torch.bfloat16, False),
    (67, 257, 8, "masks", torch.bfloat16, True), (129, 384, 6, "ties", torch.float32, False), (65, 512, 8, "masks", torch.float32, True),
    (35, 513, 8, "ties", torch.bfloat16, False), (33, 1000, 3, "masks", torch.float32, True), (9, 1024, 8, "ties", torch.float32, True),
])
def test_route_more_experts(T, E, k, kind, dtype, biased, score, normalize):
    test_route(T, E, k, kind, dtype, biased, score, normalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,kind,dtype", [
    (131, 129, 8, "masks", torch.bfloat16), (66, 256, 6, "ties", torch.float32), (35, 513, 8, "masks", torch.float32),
    (17, 1000, 5, "normal", torch.bfloat16), (9, 1024, 16, "masks", torch.bfloat16), (33, 384, 8, "ties", torch.bfloat16),
])
def test_route_gradient_more_experts(T, E, k, kind, dtype, score, normalize):
    test_route_gradient_follows_the_formula(T, E, k, kind, dtype, score, normalize)


@pytest.mark.parametrize("E,k", [(12, 8), (256, 6), (600, 16)])
def test_route_with_a_bias_that_is_not_finite(E, k):
    """+inf comes first (among several the lower index), -inf and NaN never."""
    rng = np.random.default_rng(E)
    l = logits_for(rng, 9, E, "masks")
    bias = rng.standard_normal(E).astype(np.float32)
    bias[rng.permutation(E)[:E // 2]] = -np.inf
    bias[rng.permutation(E)[:3]] = np.inf
    bias[0], bias[E - 1] = np.nan, np.inf
    for score in SCORES:
        clean, ids, w = run_route(l, k, bias, score, True, 1.0, torch.float32)
        want = R.select(clean, k, bias)
        assert np.array_equal(ids, want) and (want < 0).any() and (w[ids < 0] == 0).all()


# the element type that the cases above leave out of a shape
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [(40, 200, 8, torch.bfloat16), (33, 100, 10, torch.float32)])
def test_route_other_type(T, E, k, dtype, score):
    test_route(T, E, k, "masks", dtype, True, score, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [(20, 100, 8, torch.bfloat16), (17, 400, 8, torch.float32), (3, 2000, 8, torch.bfloat16)])
def test_route_gradient_other_type(T, E, k, dtype, score):
    test_route_gradient_follows_the_formula(T, E, k, "masks", dtype, score, False)
