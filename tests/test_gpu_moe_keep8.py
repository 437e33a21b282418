"""The experts' gated block with its checkpoint in 8 bits on the GPU, forward
and backward, against the plain 64-bit implementation and the bf16 form."""
import numpy as np
import pytest
import torch

import i8_reference as I
import moe_reference as R
from gpu_helpers import CANARY, Guarded, log
from nvfp4_block_scaled_group_amd import binding as B
from nvfp4_block_scaled_group_amd import moe
from test_gpu_moe_glu import ACTS, CASES, WIDE, case, factor, on_device, products

pytestmark = pytest.mark.gpu


def groups(f):
    return 2 * -(-f // 32)


def kept_buffers(M, f):
    return Guarded(2 * M * f, torch.int8, (M, 2 * f)), Guarded(2 * M * groups(f), torch.bfloat16, (groups(f), M))


@pytest.mark.parametrize("splits,f,k", CASES + WIDE["forward"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward(splits, f, k, kind):
    log(f"keep8 {splits} f={f} k={k} {kind}")
    rng, M, E, a, b = case(f + k + 3, splits, f, k, 2 * f)
    dev = on_device(a, b, E, 2 * f)
    h, (q, s) = Guarded(2 * M * f, torch.bfloat16, (M, f)), kept_buffers(M, f)
    moe.moe_glu_keep8(*dev, splits, h.t, q.t, s.t, act=ACTS[kind])
    plain = torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu(*dev, splits, plain, act=ACTS[kind])
    torch.cuda.synchronize()
    assert h.guards_intact() and q.guards_intact() and s.guards_intact()
    assert torch.equal(h.t, plain)
    gu, err = products(a, b, splits, 2 * f, k)
    got, step = I.kept_values(q.t, s.t, f)
    codes = q.numpy().astype(np.int64)
    assert np.abs(codes).max() <= 127
    # half a step, the products' error, and two roundings of a value of at most 127.5 steps
    assert (np.abs(got - gu) <= step * (0.5 + 128 * 4 * R.U) + err + np.abs(gu) * (step == 0)).all()
    # the scale: the group's largest magnitude over 127, rounded to bf16
    scales = s.t.double().cpu().numpy().T
    at = I.group_of(f)
    for j in range(groups(f)):
        top, off = np.abs(gu[:, at == j]).max(1), err[:, at == j].max(1)
        want = top / 127
        assert (np.abs(scales[:, j] - want) <= R.UB * want + 1.02 * off / 127 + 1e-30).all()
        zero = top + off < 2.0 ** -112
        assert (scales[zero, j] == 0).all() and (codes[zero][:, at == j] == 0).all()


def random_kept(rng, M, f, power_of_two=False):
    q = rng.integers(-127, 128, (M, 2 * f), dtype=np.int8)
    s = np.exp(rng.standard_normal((groups(f), M))) * 0.03
    s = 2.0 ** np.round(np.log2(s)) if power_of_two else s
    s[rng.random(s.shape) < 0.05] = 0.0
    return torch.from_numpy(q), R.bf16_round(s)[0]


@pytest.mark.parametrize("splits,f,k", CASES + WIDE["backward"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward(splits, f, k, kind):
    log(f"keep8 bwd {splits} f={f} k={k} {kind}")
    rng, M, E, a, b = case(f + k + 4, splits, f, k, f)
    dev = on_device(a, b, E, f)
    q, s = random_kept(rng, M, f)
    gu, _ = I.kept_values(q, s, f)
    dh, err = products(a, b, splits, f, k)
    out, again = Guarded(4 * M * f, torch.bfloat16, (M, 2 * f)), Guarded(2 * M * f, torch.bfloat16, (M, f))
    moe.moe_glu_bwd_keep8(*dev, splits, q.to("cuda:0"), s.to("cuda:0"), out.t, h=again.t, act=ACTS[kind])
    alone = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_bwd_keep8(*dev, splits, q.to("cuda:0"), s.to("cuda:0"), alone, act=ACTS[kind])
    torch.cuda.synchronize()
    assert out.guards_intact() and again.guards_intact() and torch.equal(out.t, alone)
    g, u = gu[:, :f], gu[:, f:]
    v, d = R.act(g, kind)
    rel = R.act_rel(g, kind)
    # a kept value is exact in fp32, so the errors are those of the bf16 form
    want = np.concatenate([dh * u * d, dh * v], 1)
    slope = rel * (np.abs(d) + 1) + np.abs(v) * 8 * R.U * (1 + g ** 2)
    eg = err * np.abs(u) * (np.abs(d) + slope) + np.abs(dh * u) * (slope + 8 * R.U)
    eu = err * np.abs(v) * (1 + rel) + np.abs(dh * v) * (rel + 8 * R.U)
    e = np.concatenate([eg, eu], 1) + 1e-30
    R.check(out.t, want, e + R.UB * (np.abs(want) + e), "dgu")
    R.check(again.t, v * u, R.glu_bound(g, u, 0 * g, 0 * u, kind), "h")


@pytest.mark.parametrize("splits,f,k", [CASES[3], WIDE["backward"][0]])
def test_backward_equals_the_bf16_form_on_values_that_both_hold(splits, f, k):
    rng, M, E, a, b = case(6, splits, f, k, f)
    dev = on_device(a, b, E, f)
    q, s = random_kept(rng, M, f, power_of_two=True)
    gu = torch.from_numpy(I.kept_values(q, s, f)[0]).to(torch.bfloat16).to("cuda:0")
    got, want = (torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    moe.moe_glu_bwd_keep8(*dev, splits, q.to("cuda:0"), s.to("cuda:0"), got)
    moe.moe_glu_bwd(*dev, splits, gu, want)
    assert torch.equal(got, want)


def test_backward_at_the_largest_scale():
    """S = 2^121: 127 S is finite, 128 S is not; dh is small enough for finite gradients."""
    splits, f, k = [128, 256], 208, 128
    rng, M, E, a, b = case(8, splits, f, k, f)
    a[2][:] *= np.float32(2.0 ** -100)
    dev = on_device(a, b, E, f)
    q, s = random_kept(rng, M, f)
    s[:] = 2.0 ** 121
    gu = torch.from_numpy(I.kept_values(q, s, f)[0]).to(torch.bfloat16).to("cuda:0")
    got, want = (torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    moe.moe_glu_bwd_keep8(*dev, splits, q.to("cuda:0"), s.to("cuda:0"), got)
    moe.moe_glu_bwd(*dev, splits, gu, want)
    assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_follows_differences(kind):
    """dh is exact here; the loss sum(dh * act(g) * u) is differenced in 64 bits at the kept values."""
    rng = np.random.default_rng(2)
    f, k, M = 48, 128, 128
    a = (np.full((M, k // 2), 0x22, np.uint8), np.full((M, k // 16), 0x38, np.uint8), np.full(M, 2688, np.float32))
    b = (rng.integers(0, 3, (f, k // 2), dtype=np.uint8) * 2, np.full((f, k // 16), 0x38, np.uint8), np.full(f, 2688, np.float32))
    q, s = random_kept(rng, M, f)
    gu, _ = I.kept_values(q, s, f)
    out = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_bwd_keep8(*on_device(a, b, 1, f), [M], q.to("cuda:0"), s.to("cuda:0"), out, act=ACTS[kind])
    dh, _ = R.product(R.decode(*a[:2]), factor(a[2]), R.decode(*b[:2]), factor(b[2]))
    eps, num = 1e-5, np.empty((M, 2 * f))
    for c in range(2):
        d = np.zeros((M, 2 * f))
        d[:, c * f:(c + 1) * f] = eps
        up, down = gu + d, gu - d
        num[:, c * f:(c + 1) * f] = dh * (R.act(up[:, :f], kind)[0] * up[:, f:] - R.act(down[:, :f], kind)[0] * down[:, f:]) / (2 * eps)
    R.check(out, num, R.UB * np.abs(num) * 1.01 + 1e-5 * (1 + np.abs(dh).max()) * (1 + np.abs(gu).max()), "dgu")


def test_a_step_through_the_checkpoint():
    """Forward, then backward on what it kept: near the bf16 form's gradients, by the size of the steps."""
    splits, f, k, kd = [256, 0, 384], 208, 256, 384
    rng, M, E, a, b = case(31, splits, f, k, 2 * f)
    _, _, _, da, db = case(32, splits, f, kd, f)
    fwd, bwd = on_device(a, b, E, 2 * f), on_device(da, db, E, f)
    h, again = (torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    kept, d8 = moe.alloc_keep8(M, f), torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_keep8(*fwd, splits, h, **kept)
    moe.moe_glu_bwd_keep8(*bwd, splits, **kept, dgu=d8, h=again)
    gu, _ = products(a, b, splits, 2 * f, k)
    got, _ = I.kept_values(kept["gu8"], kept["gu_scale"], f)
    dh, err = products(da, db, splits, f, kd)
    g, u = got[:, :f], got[:, f:]
    v, d = R.act(g, "silu")
    want = np.concatenate([dh * u * d, dh * v], 1)
    mag = np.concatenate([err * np.abs(u) * 1.2 + np.abs(dh * u) * 64 * R.U, (err + np.abs(dh) * 64 * R.U) * (np.abs(v) + 1)], 1)
    R.check(d8, want, mag * 2 + R.UB * np.abs(want) * 1.01 + 1e-30, "dgu")
    assert np.abs(got - gu).max() <= np.abs(gu).max() / 127 * 0.51


def test_groups_that_are_no_numbers_or_nothing():
    splits, f, k = [256], 80, 128
    rng, M, E, a, b = case(9, splits, f, k, 2 * f)
    a[2][:] = 1.0
    a[2][3], a[2][5], a[2][7], a[2][9] = np.inf, 0.0, 1e-36, np.nan
    b[2][:] = 1.0
    b[2][40] = np.inf                                # gate column 40: group 1 of g, every row
    b[2][f:f + 16] = 1e-3
    dev = on_device(a, b, E, 2 * f)
    h, kept = torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0"), moe.alloc_keep8(M, f)
    moe.moe_glu_keep8(*dev, splits, h, **kept)
    s, q = kept["gu_scale"].float().cpu().numpy(), kept["gu8"].cpu().numpy()
    bad = np.zeros((groups(f), M), bool)
    bad[:, 3] = bad[:, 9] = True
    bad[1, :] = True
    assert np.array_equal(np.isnan(s), bad)
    at = I.group_of(f)
    assert (q[bad.T[:, at]] == 0).all()
    assert (s[:, 5][~bad[:, 5]] == 0).all() and (q[5] == 0).all() and (s[:, 7][~bad[:, 7]] == 0).all() and (q[7] == 0).all()
    # a scale that is no number reaches its own group's gradients alone
    _, _, _, da, db = case(10, splits, f, k, f)
    d, again = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0"), torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_bwd_keep8(*on_device(da, db, E, f), splits, **kept, dgu=d, h=again)
    nan = torch.isnan(again).cpu().numpy()
    gbad, ubad = bad.T[:, at[:f]], bad.T[:, at[f:]]
    assert np.array_equal(nan, gbad | ubad)
    assert np.isfinite(d.float().cpu().numpy()[~np.concatenate([gbad | ubad, gbad], 1)]).all()


@pytest.mark.parametrize("splits,f,k,spare", [([128, 0, 256], 48, 256, 256), (*WIDE["forward"][0], 640)])
def test_device_routing_writes_the_routed_rows_alone(splits, f, k, spare):
    rng, M, E, a, b = case(17, splits, f, k, 2 * f)
    _, _, _, da, db = case(18, splits, f, k, f)
    cap = M + spare
    pad = lambda o: [np.concatenate([v, np.full((spare, *v.shape[1:]), 0x7F, v.dtype)]) for v in o]  # noqa: E731
    fwd, bwd = on_device(pad(a), b, E, 2 * f), on_device(pad(da), db, E, f)
    h, again, d = (Guarded(2 * cap * w, torch.bfloat16, (cap, w)) for w in (f, f, 2 * f))
    q, s = kept_buffers(cap, f)
    status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    offs = torch.tensor(B.offsets_from_splits(splits), dtype=torch.int32, device="cuda:0")
    moe.moe_glu_keep8_graphsafe(*fwd, offs, h.t, q.t, s.t, status)
    moe.moe_glu_bwd_keep8_graphsafe(*bwd, offs, q.t, s.t, d.t, status, h=again.t)
    kept = moe.alloc_keep8(M, f)
    wh, wagain, wd = (torch.empty((M, w), dtype=torch.bfloat16, device="cuda:0") for w in (f, f, 2 * f))
    moe.moe_glu_keep8(*on_device(a, b, E, 2 * f), splits, wh, **kept)
    moe.moe_glu_bwd_keep8(*on_device(da, db, E, f), splits, **kept, dgu=wd, h=wagain)
    torch.cuda.synchronize()
    assert int(status) == 0 and all(g.guards_intact() for g in (h, again, d, q, s))
    for got, want in ((h.t[:M], wh), (again.t[:M], wagain), (d.t[:M], wd), (q.t[:M], kept["gu8"]),
                      (s.t[:, :M], kept["gu_scale"])):
        assert torch.equal(got, want)
    for rest in (h.t[M:], again.t[M:], d.t[M:], q.t[M:], s.t[:, M:]):
        assert (rest.contiguous().view(torch.uint8) == CANARY).all()
    for bad, bit in (([100] + [M] * (E - 1), B.NVFP4G_DEV_UNALIGNED), ([M, 0] + [M] * (E - 2), B.NVFP4G_DEV_NONMONO),
                     ([0] * (E - 1) + [cap + 128], B.NVFP4G_DEV_OVERFLOW)):
        h, (q, s) = Guarded(2 * cap * f, torch.bfloat16, (cap, f)), kept_buffers(cap, f)
        status.zero_()
        moe.moe_glu_keep8_graphsafe(*fwd, torch.tensor(bad, dtype=torch.int32, device="cuda:0"), h.t, q.t, s.t, status)
        torch.cuda.synchronize()
        assert int(status) & bit
        for g in (h, q, s):
            assert (g.t.contiguous().view(torch.uint8) == CANARY).all()


# rows and columns whose tiles are the wide ones (128 columns forward, 256
# backward), the last column of them ragged: 510 of them, and 768 (more than 512:
# their XCD order); compared with the bf16 form, whose tests hold it to 64 bits
WIDE8 = {"forward": [([4096, 0, 6784], 656), ([8192, 128, 8064], 752)],
         "backward": [([4096, 0, 6784], 1296), ([8192, 128, 8064], 1520)]}


@pytest.mark.parametrize("at", [0, 1])
def test_forward_wide_tiles(at):
    (splits, f), k = WIDE8["forward"][at], 256
    assert sum(splits) // 128 * -(-f // 128) == (510, 768)[at]
    rng, M, E, a, b = case(f, splits, f, k, 2 * f)
    dev = on_device(a, b, E, 2 * f)
    h, plain = Guarded(2 * M * f, torch.bfloat16, (M, f)), torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0")
    (q, s), gu = kept_buffers(M, f), torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_keep8(*dev, splits, h.t, q.t, s.t)
    moe.moe_glu(*dev, splits, plain, gu=gu)
    torch.cuda.synchronize()
    assert h.guards_intact() and q.guards_intact() and s.guards_intact() and torch.equal(h.t, plain)
    step = s.t.float().t()[:, torch.from_numpy(I.group_of(f)).to("cuda:0")]
    got = q.t.float() * step
    # half a step, and the rounding of the bf16 value it is compared with (2^-8 of it, with room for fp32 here)
    assert ((got - gu.float()).abs() <= step * 0.501 + gu.float().abs() * 1.01 * R.UB).all()


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_wide_tiles(at, kind):
    (splits, f), k = WIDE8["backward"][at], 256
    assert sum(splits) // 128 * -(-f // 256) == (510, 768)[at]
    rng, M, E, a, b = case(f, splits, f, k, f)
    dev = on_device(a, b, E, f)
    q, s = random_kept(rng, M, f, power_of_two=True)
    q, s = q.to("cuda:0"), s.to("cuda:0")
    gu = (q.float() * s.float().t()[:, torch.from_numpy(I.group_of(f)).to("cuda:0")]).to(torch.bfloat16)
    out, again = Guarded(4 * M * f, torch.bfloat16, (M, 2 * f)), Guarded(2 * M * f, torch.bfloat16, (M, f))
    want = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_glu_bwd_keep8(*dev, splits, q, s, out.t, h=again.t, act=ACTS[kind])
    moe.moe_glu_bwd(*dev, splits, gu, want, act=ACTS[kind])
    torch.cuda.synchronize()
    assert out.guards_intact() and again.guards_intact() and torch.equal(out.t, want)
    rows = rng.choice(M, 300, replace=False)
    at64 = gu[torch.from_numpy(rows).to("cuda:0")].double().cpu().numpy()
    g, u = at64[:, :f], at64[:, f:]
    R.check(again.t[torch.from_numpy(rows).to("cuda:0")], R.act(g, kind)[0] * u, R.glu_bound(g, u, 0 * g, 0 * u, kind), "h")


def test_codes_are_the_nearest_to_the_quotient():
    """g and u that are exact in the kernel, at and beside the ties between two codes and at scales that are themselves
    ties between two bf16 values: the code is the whole number nearest to the fp32 quotient, ties to even, and a
    group's largest is +-127."""
    G, k, M = 64, 128, 128
    f, rng, F32 = 32 * G, np.random.default_rng(4), np.float32
    want = np.empty((2 * G, 32))                       # [group of g then u, column]
    for j in range(2 * G):
        e, top = int(rng.integers(-40, 40)), 1 + int(rng.integers(0, 128)) / 128
        top += (0, 1, -1)[j % 3] / 256                 # max / 127: a bf16 value, or half way to the next or the last one
        step = float(torch.tensor(top * 2.0 ** e, dtype=torch.float64).to(torch.bfloat16))
        ties = ((rng.integers(0, 126, 31) + 0.5) * step).astype(F32)              # 16 bits: exact
        beside = np.nextafter(ties, F32(np.inf) * rng.choice([-1, 1], 31).astype(F32))
        want[j, 0], want[j, 1:] = 127 * top * 2.0 ** e, np.where(rng.random(31) < 0.6, ties, beside)
    # a line's value is amax / 2688 in fp32: the amax that gives the wanted one, or one beside it
    want = want.reshape(-1).astype(F32)
    amax = (want.astype(np.float64) * 2688).astype(F32)
    for near in (np.nextafter(amax, F32(np.inf)), np.nextafter(amax, F32(0))):
        amax = np.where((amax / F32(2688) != want) & (near / F32(2688) == want), near, amax)
    v = (amax / F32(2688)).reshape(2 * G, 32)
    one = np.zeros((2 * f, k // 2), np.uint8)
    one[:, 0] = 0x02                                   # 1.0, then zeros
    rows = np.zeros((M, k // 2), np.uint8)
    rows[:, 0] = np.where(np.arange(M) % 2, 0x0A, 0x02)  # -1.0 in the odd rows
    a = (rows, np.full((M, k // 16), 0x38, np.uint8), np.full(M, 2688, F32))
    b = (one, np.full((2 * f, k // 16), 0x38, np.uint8), amax)
    h, kept = torch.empty((M, f), dtype=torch.bfloat16, device="cuda:0"), moe.alloc_keep8(M, f)
    moe.moe_glu_keep8(*on_device(a, b, 1, 2 * f), [M], h, **kept)
    s = torch.from_numpy(np.abs(v).max(1) / F32(127)).to(torch.bfloat16)
    codes = np.rint(v / s.float().numpy()[:, None]).astype(np.int64).reshape(-1)
    got, scale = kept["gu8"].cpu().numpy().astype(np.int64), kept["gu_scale"].cpu()
    assert torch.equal(scale, s[:, None].expand(2 * G, M))
    # the cases do what they are for: exact ties, and ties of the scale
    assert (np.abs(v / s.float().numpy()[:, None] % 1) == 0.5).sum() > 500
    assert (np.abs(codes.reshape(-1, 32)[:, 0]) == 127).all()
    for r in range(M):
        assert np.array_equal(got[r], -codes if r % 2 else codes), (r, np.nonzero(got[r] != (-codes if r % 2 else codes))[0][:5])
