"""Low-rank adapters of many requests beside a shared NVFP4 projection on the
GPU, against the plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import moe_reference as R
from gpu_helpers import Guarded, log
from nvfp4_block_scaled_group_amd import moe

pytestmark = pytest.mark.gpu


def make(seed, T, N, K, r, A):
    rng = np.random.default_rng(seed)
    w = R.random_lines(rng, N, K, big=8.0 / K)
    xt, x = R.bf16_round(rng.standard_normal((T, K)))
    at, a = R.bf16_round(rng.standard_normal((A, r, K)) * K ** -0.5)
    bt, b = R.bf16_round(rng.standard_normal((A, N, r)))
    alpha = rng.standard_normal(A).astype(np.float32)
    return rng, w, xt, x, at, a, bt, b, alpha


def call(w, xt, at, bt, ids, alpha, T, N, K, r):
    y = Guarded(2 * T * N, torch.bfloat16, (T, N))
    ws = torch.full((max(16, moe.lora_workspace(T, K, N, r)),), 0xFF, dtype=torch.uint8, device="cuda:0")  # NaN patterns
    moe.lora_linear(xt.to("cuda:0"), *[R.to_dev(v) for v in w], at.to("cuda:0"), bt.to("cuda:0"),
                    R.to_dev(ids.astype(np.int32)), R.to_dev(alpha), y.t, ws)
    torch.cuda.synchronize()
    assert y.guards_intact()
    return y.t


def expect(w, x, a, b, ids, alpha, K, r):
    xw, f = R.decode(*w[:2]), w[2].astype(np.float64) / 2688
    y, mag = (x @ xw.T) * f, (np.abs(x) @ np.abs(xw).T) * f
    err = R.gemm_bound(mag, K)
    for t, i in enumerate(ids):
        if 0 <= i < a.shape[0]:
            v, va = a[i] @ x[t], np.abs(a[i]) @ np.abs(x[t])
            y[t] += alpha[i] * (b[i] @ v)
            # fp32 sums over K and over the rank; v (or its two bf16 halves, 2^-18) and alpha rounded
            err[t] += abs(alpha[i]) * (np.abs(b[i]) @ (((2 * K + 8) * R.U) * va + (2 * r + 8) * R.U * np.abs(v) + 2.0 ** -17 * np.abs(v)))
    err = err + (np.abs(y) + err) * 4 * R.U
    return y, err + R.UB * (np.abs(y) + err) + 1e-30


SHAPES = [  # T, N, K, rank, adapters
    (1, 16, 32, 8, 1), (3, 48, 96, 16, 2), (16, 272, 256, 24, 5), (17, 64, 1056, 40, 3), (33, 32, 128, 64, 40),
    (64, 80, 544, 128, 7), (65, 16, 32, 8, 3), (130, 272, 96, 16, 4), (257, 528, 288, 24, 300), (300, 48, 2080, 128, 2),
    (8, 512, 7168, 16, 6), (200, 256, 64, 32, 1),
]


@pytest.mark.parametrize("T,N,K,r,A", SHAPES)
@pytest.mark.parametrize("mix", ["any", "runs", "none", "one"])
def test_lora(T, N, K, r, A, mix):
    log(f"lora T={T} N={N} K={K} r={r} A={A} {mix}")
    rng, w, xt, x, at, a, bt, b, alpha = make(T + K, T, N, K, r, A)
    if mix == "any":
        ids = rng.integers(-2, A + 1, T)            # ids on both sides of the range
    elif mix == "runs":
        ids = np.sort(rng.integers(-1, A, T))
    elif mix == "none":
        ids = np.full(T, -1)
    else:
        ids = np.full(T, A - 1)
    got = call(w, xt, at, bt, ids, alpha, T, N, K, r)
    want, err = expect(w, x, a, b, ids, alpha.astype(np.float64), K, r)
    R.check(got, want, err, "y")


def test_an_adapter_that_overflows_stays_in_its_rows():
    T, N, K, r, A = 130, 64, 128, 16, 3
    rng, w, xt, x, at, a, bt, b, alpha = make(4, T, N, K, r, A)
    ids = rng.integers(0, 3, T)
    ref = call(w, xt, at, bt, ids, alpha, T, N, K, r).clone()
    at[1] = float("nan")
    bt[1] = float("inf")
    for rows in (T, 40):
        got = call(w, xt[:rows], at, bt, ids[:rows], alpha, rows, N, K, r)
        keep = torch.from_numpy(ids[:rows] != 1).to("cuda:0")
        assert torch.isfinite(got[keep].float()).all()
        if rows == T:
            assert torch.equal(got[keep], ref[keep])
        assert torch.isnan(got[~keep].float()).all()


def test_results_do_not_depend_on_the_run():
    T, N, K, r, A = 48, 256, 2048, 32, 9
    rng, w, xt, x, at, a, bt, b, alpha = make(5, T, N, K, r, A)
    ids = rng.integers(-1, A, T)
    first = call(w, xt, at, bt, ids, alpha, T, N, K, r).clone()
    for _ in range(3):
        assert torch.equal(call(w, xt, at, bt, ids, alpha, T, N, K, r), first)


def test_offsets_past_32_bits():
    """Rows of x and y beyond 4 GiB."""
    K, N, r, A = 8192, 16, 8, 1
    T = (1 << 32) // (2 * K) + 200
    rng, w, _, _, at, a, bt, b, alpha = make(6, 1, N, K, r, A)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda:0")
    rows = [0, 1, T - 130, T - 1]
    vt, v = R.bf16_round(rng.standard_normal((len(rows), K)))
    x[rows] = vt.to("cuda:0")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0")
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda:0")
    ids[rows] = 0
    ws = torch.empty(moe.lora_workspace(T, K, N, r), dtype=torch.uint8, device="cuda:0")
    moe.lora_linear(x, *[R.to_dev(t) for t in w], at.to("cuda:0"), bt.to("cuda:0"), ids, R.to_dev(alpha), y, ws)
    torch.cuda.synchronize()
    want, err = expect(w, v, a, b, [0] * len(rows), alpha.astype(np.float64), K, r)
    R.check(y[rows], want, err, "y")
    assert float(y.float().abs().sum()) == float(y[rows].float().abs().sum())


FORMS = [  # T, N, K, rank, adapters
    (1030, 11024, 64, 24, 9),    # whole wide tiles, over the end of a window of row order
    (2100, 48, 96, 16, 50),      # half as wide tiles, three windows
    (100, 48, 4160, 40, 28),     # parts of the contraction, rows in order, an adapter in every other row
    (140, 272, 1312, 128, 3),
    (32, 1040, 4128, 72, 32),    # every row of the first form, more than one chunk of x, ranks past one load
]


@pytest.mark.parametrize("T,N,K,r,A", FORMS)
def test_lora_forms(T, N, K, r, A):
    log(f"lora T={T} N={N} K={K} r={r} A={A}")
    rng, w, xt, x, at, a, bt, b, alpha = make(T + K + 1, T, N, K, r, A)
    ids = rng.integers(-1, A, T)
    got = call(w, xt, at, bt, ids, alpha, T, N, K, r)
    want, err = expect(w, x, a, b, ids, alpha.astype(np.float64), K, r)
    R.check(got, want, err, "y")


@pytest.mark.parametrize("T,N,K", [
    (8, 48, 96),          # few rows
    (40, 48, 96),         # half as wide tiles
    (40, 48, 1056),       # parts of the contraction
    (1030, 11024, 96),    # wide tiles
])
def test_a_scale_that_is_not_a_number_stays_in_its_line(T, N, K):
    """K is an odd multiple of 32: the last contraction step of a line reaches
    the scales of the next one."""
    log(f"lora NaN scale T={T} N={N} K={K}")
    r, A = 8, 1
    rng, w, xt, x, at, a, bt, b, alpha = make(9, T, N, K, r, A)
    ids = np.full(T, -1)
    ref = call(w, xt, at, bt, ids, alpha, T, N, K, r).clone()
    bad = [1, 17, N - 1]                    # lines with a first and a second block that are no numbers
    w[1][bad, 0], w[1][bad, 1] = 0x7F, 0xFF
    got = call(w, xt, at, bt, ids, alpha, T, N, K, r)
    keep = torch.ones(N, dtype=torch.bool, device="cuda:0")
    keep[bad] = False
    assert torch.equal(got[:, keep], ref[:, keep])
    assert torch.isnan(got[:, ~keep].float()).all()


@pytest.mark.parametrize("T,N,K", [
    (8, 16, 64),          # few rows
    (40, 16, 64),         # half as wide tiles
    (40, 16, 1024),       # parts of the contraction
    (1030, 11024, 64),    # wide tiles
])
def test_inner_product_is_kept_in_fp32(T, N, K):
    """Two inner products that differ in their twentieth bit, with factors 1
    and -1 (every other sum on the way is exact); and a scaled inner product
    above bf16's largest value whose factor brings it back into range."""
    log(f"lora fp32 inner product T={T} N={N} K={K}")
    r = 8
    w = (np.zeros((N, K // 2), np.uint8), np.full((N, K // 16), 0x38, np.uint8), np.ones(N, np.float32))
    x, a, b = torch.zeros((T, K)), torch.zeros((2, r, K)), torch.zeros((2, N, r))
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -20
    a[0, 0, :3] = 1.0
    a[0, 1, :2] = 1.0
    b[0, :, 0], b[0, :, 1] = 1.0, -1.0
    a[1, 0, 0], b[1, :, 0] = 1.0, 2.0 ** -100
    alpha = np.array([1.0, R.FLT_MAX], np.float32)
    ids = np.arange(T) % 3 - 1
    got = call(w, *(t.to(torch.bfloat16) for t in (x, a, b)), ids, alpha, T, N, K, r)
    want = torch.tensor([0.0, 2.0 ** -20, R.FLT_MAX * 2.0 ** -100], dtype=torch.float64)
    want = want.to(torch.bfloat16)[torch.from_numpy(ids + 1)].to("cuda:0")
    assert torch.equal(got, want[:, None].expand(T, N))


def test_a_workspace_serves_smaller_batches_and_ranks():
    """One workspace, sized for the largest batch and rank, for every smaller
    one and for no adapters."""
    N, K, r = 528, 2048, 16
    rng, w, xt, x, at, a, bt, b, alpha = make(12, 600, N, K, r, 2)
    ids = rng.integers(-1, 2, 600)
    dev = [R.to_dev(v) for v in w]
    ws = torch.empty(moe.lora_workspace(20000, K, N, r), dtype=torch.uint8, device="cuda:0")
    for T in (1, 33, 100, 128, 400, 600):
        for rank, adapters in ((r, 2), (8, 2), (r, 0)):
            y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0")
            la, lb = at[:adapters, :rank].contiguous(), bt[:adapters, :, :rank].contiguous()
            moe.lora_linear(xt[:T].to("cuda:0"), *dev, la.to("cuda:0"), lb.to("cuda:0"), R.to_dev(ids[:T].astype(np.int32)),
                            R.to_dev(alpha[:adapters]), y, ws)
            torch.cuda.synchronize()
            la64, lb64 = la.double().numpy(), lb.double().numpy()
            want, err = expect(w, x[:T], la64, lb64, ids[:T], alpha.astype(np.float64), K, rank)
            R.check(y, want, err, f"y of {T} rows, rank {rank}, {adapters} adapters")


@pytest.mark.parametrize("T,N,K", [(5, 48, 192), (5, 48, 96), (40, 48, 192), (40, 48, 1056)])
def test_scales_on_any_dword(T, N, K):
    log(f"lora scales on a dword T={T} N={N} K={K}")
    r, A = 8, 2
    rng, w, xt, x, at, a, bt, b, alpha = make(13, T, N, K, r, A)
    ids = rng.integers(-1, A, T)
    ref = call(w, xt, at, bt, ids, alpha, T, N, K, r)
    room = torch.full((w[1].size + 16,), 0x7F, dtype=torch.uint8, device="cuda:0")
    scale = room[4:4 + w[1].size].view(w[1].shape)
    scale.copy_(R.to_dev(w[1]))
    assert scale.data_ptr() % 16 == 4
    y = torch.empty_like(ref)
    ws = torch.empty(moe.lora_workspace(T, K, N, r), dtype=torch.uint8, device="cuda:0")
    moe.lora_linear(xt.to("cuda:0"), R.to_dev(w[0]), scale, R.to_dev(w[2]), at.to("cuda:0"), bt.to("cuda:0"),
                    R.to_dev(ids.astype(np.int32)), R.to_dev(alpha), y, ws)
    assert torch.equal(y, ref)


MORE_FORMS = [  # T, N, K, rank, adapters
    (1030, 11024, 288, 72, 5),    # wide tiles, five steps of which the last is half, ranks past 64
    (1030, 11024, 160, 16, 1),    # the same with one adapter: rows as they come
    (300, 528, 352, 104, 6),      # half as wide tiles, six steps, ranks past 64
    (150, 272, 416, 128, 1),
]


@pytest.mark.parametrize("T,N,K,r,A", MORE_FORMS)
def test_lora_more_forms(T, N, K, r, A):
    test_lora_forms(T, N, K, r, A)


@pytest.mark.parametrize("T,N,K", [(5, 48, 96), (20, 272, 544), (40, 144, 96), (40, 144, 1056), (1030, 11024, 96)])
def test_projection_alone(T, N, K):
    """No adapters: through the binding with empty tensors, and from C with
    NULL pointers, which give the same bits."""
    log(f"lora without adapters T={T} N={N} K={K}")
    rng, w, xt, x, *_ = make(14, T, N, K, 8, 1)
    xd, wd = xt.to("cuda:0"), [R.to_dev(v) for v in w]
    y, again = Guarded(2 * T * N, torch.bfloat16, (T, N)), Guarded(2 * T * N, torch.bfloat16, (T, N))
    size = moe.lora_workspace(T, K, N, 0)
    ws = torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device="cuda:0")
    none = torch.empty((0, 8, K), dtype=torch.bfloat16, device="cuda:0"), torch.empty((0, N, 8), dtype=torch.bfloat16, device="cuda:0")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda:0")       # no adapter has this number
    moe.lora_linear(xd, *wd, *none, ids, torch.empty(0, device="cuda:0"), y.t, ws)
    rc = moe.load_library().lora_linear(xd.data_ptr(), T, K, *[t.data_ptr() for t in wd], N, None, None, None, 0, 0, None,
                                        again.t.data_ptr(), ws.data_ptr() if size else None, size,
                                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and y.guards_intact() and again.guards_intact() and torch.equal(y.t, again.t)
    want, err = expect(w, x, np.zeros((0, 8, K)), np.zeros((0, N, 8)), [-1] * T, np.zeros(0), K, 8)
    R.check(y.t, want, err, "y")
