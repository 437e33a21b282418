"""Tokens into packed rows and back on the GPU (moe_dispatch, moe_combine) and
their gradients, against the plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import moe_reference as R
from gpu_helpers import CANARY, Guarded, log
from nvfp4_block_scaled_group_amd import moe

pytestmark = pytest.mark.gpu


def choices(rng, T, E, k, holes=0.1):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), np.int64)
    ids[rng.random(ids.shape) < holes] = -1
    if T > 2:
        ids[1] = -1                       # a token without any expert
    return ids.astype(np.int32)


def planned(rng, T, E, k, spare=128):
    ids = choices(rng, T, E, k)
    need = int(R.plan(ids, E, 0)[1][-1])
    cap = need + spare
    counts, ends, rows, src = R.plan(ids, E, cap)
    return cap, need, rows.reshape(T, k).astype(np.int32), src.astype(np.int32), ends.astype(np.int32)


SHAPES = [(0, 4, 2, 16), (1, 1, 1, 16), (3, 8, 2, 48), (65, 8, 3, 528), (33, 64, 6, 2064), (130, 20, 16, 256), (40, 9, 8, 7168)]


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch(T, E, k, H, weighted):
    log(f"dispatch T={T} E={E} k={k} H={H} {weighted}")
    rng = np.random.default_rng(T + H)
    cap, need, rows, src, ends = planned(rng, T, E, k)
    xt, x = R.bf16_round(rng.standard_normal((T, H)))
    w = rng.random((T, k)).astype(np.float32)
    w[rows < 0] = np.nan                   # a weight without a row is not used
    out = Guarded(2 * cap * H, torch.bfloat16, (cap, H))
    moe.moe_dispatch(xt.to("cuda:0"), R.to_dev(rows), R.to_dev(src), R.to_dev(ends), out.t,
                     weights=R.to_dev(w) if weighted else None)
    torch.cuda.synchronize()
    assert out.guards_intact()
    want = np.zeros((cap, H))
    t, j = np.nonzero(rows >= 0)
    want[rows[t, j]] = x[t] * (w[t, j].astype(np.float64)[:, None] if weighted else 1.0)
    # the fp32 product and its rounding to bf16
    R.check(out.t[:need], want[:need], (R.UB + 2 * R.U) * np.abs(want[:need]) if weighted else 0.0, "out")
    raw = out.t[need:].contiguous().view(torch.uint8).cpu().numpy()
    assert (raw == CANARY).all()           # rows past the last group stay as they were


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_combine_and_its_gradient(T, E, k, H, kind):
    log(f"combine T={T} E={E} k={k} H={H} {kind}")
    rng = np.random.default_rng(T + H + 1)
    cap, need, rows, src, ends = planned(rng, T, E, k)
    y32 = rng.standard_normal((cap, H)).astype(np.float32)
    yt, y = R.bf16_round(y32) if kind == "bf16" else (torch.from_numpy(y32), y32.astype(np.float64))
    yt = yt.clone()
    unused = np.ones(cap, bool)
    unused[rows[rows >= 0]] = False
    yt[torch.from_numpy(unused)] = float("nan")    # padding rows are never read
    yd = yt.to("cuda:0")
    w = rng.random((T, k)).astype(np.float32)
    on = rows >= 0
    t, j = np.nonzero(on)
    for weighted in (True, False):
        out = Guarded(2 * T * H, torch.bfloat16, (T, H))
        moe.moe_combine(yd, R.to_dev(rows), out.t, weights=R.to_dev(w) if weighted else None)
        torch.cuda.synchronize()
        assert out.guards_intact()
        f = w.astype(np.float64) if weighted else np.ones((T, k))
        want, mag = np.zeros((T, H)), np.zeros((T, H))
        np.add.at(want, t, f[t, j][:, None] * y[rows[t, j]])
        np.add.at(mag, t, f[t, j][:, None] * np.abs(y[rows[t, j]]))
        # k fused products and sums in fp32, one rounding to bf16
        R.check(out.t, want, (k + 1) * R.U * mag + R.UB * (np.abs(want) + k * R.U * mag), "out")
    dt, d = R.bf16_round(rng.standard_normal((T, H)))
    dy, dw = Guarded(2 * cap * H, torch.bfloat16, (cap, H)), Guarded(4 * T * k, torch.float32, (T, k))
    moe.moe_dispatch(dt.to("cuda:0"), R.to_dev(rows), R.to_dev(src), R.to_dev(ends), dy.t, weights=R.to_dev(w), y=yd,
                     dweights=dw.t)
    torch.cuda.synchronize()
    assert dy.guards_intact() and dw.guards_intact()
    want = np.zeros((cap, H))
    want[rows[t, j]] = d[t] * w.astype(np.float64)[t, j][:, None]
    R.check(dy.t[:need], want[:need], (R.UB + 2 * R.U) * np.abs(want[:need]), "dy")
    wdw, mag = np.zeros((T, k)), np.zeros((T, k))
    wdw[t, j] = (d[t] * y[rows[t, j]]).sum(1)
    mag[t, j] = np.abs(d[t] * y[rows[t, j]]).sum(1)
    # a lane adds at most H / 256 fused products, then 6 + 3 additions across lanes and waves
    R.check(dw.t, wdw, (H / 256 + 8 + 10) * R.U * mag, "dweights")


def test_dispatch_is_the_transpose_of_combine():
    """<dispatch(x), y> == <x, combine(y)> without weights, on integers (exact
    in every format on the way)."""
    rng = np.random.default_rng(5)
    T, E, k, H = 37, 6, 3, 64
    cap, need, rows, src, ends = planned(rng, T, E, k, spare=0)
    x = torch.from_numpy(rng.integers(-4, 5, (T, H)).astype(np.float32)).to(torch.bfloat16).to("cuda:0")
    y = torch.from_numpy(rng.integers(-4, 5, (cap, H)).astype(np.float32)).to("cuda:0")
    p, c = torch.empty((cap, H), dtype=torch.bfloat16, device="cuda:0"), torch.empty((T, H), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_dispatch(x, R.to_dev(rows), R.to_dev(src), R.to_dev(ends), p)
    moe.moe_combine(y, R.to_dev(rows), c)
    assert float((p.double() * y.double()).sum()) == float((x.double() * c.double()).sum())


def test_combine_gradient_follows_differences():
    """The loss is linear in y and in the weights, so a difference of any size
    gives the gradient up to the rounding of the bf16 outputs."""
    rng = np.random.default_rng(6)
    T, E, k, H = 6, 4, 2, 32
    cap, need, rows, src, ends = planned(rng, T, E, k, spare=0)
    y = rng.standard_normal((cap, H)).astype(np.float32)
    w = rng.random((T, k)).astype(np.float32)
    dt, d = R.bf16_round(rng.standard_normal((T, H)))
    dy, dw = torch.zeros((cap, H), dtype=torch.bfloat16, device="cuda:0"), torch.empty((T, k), device="cuda:0")
    moe.moe_dispatch(dt.to("cuda:0"), R.to_dev(rows), R.to_dev(src), R.to_dev(ends), dy, weights=R.to_dev(w),
                     y=R.to_dev(y), dweights=dw)

    def loss(yy, ww):
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda:0")
        moe.moe_combine(R.to_dev(yy.astype(np.float32)), R.to_dev(rows), out, weights=R.to_dev(ww.astype(np.float32)))
        return out.double().cpu().numpy()

    base = loss(y, w)
    for t in range(T):
        for j in range(k):
            if rows[t, j] < 0:
                assert float(dw[t, j]) == 0
                continue
            step = 64.0
            w2 = w.copy()
            w2[t, j] += step
            up = loss(y, w2)
            num = ((up - base) * d).sum() / step
            err = (np.abs(up[t]) + np.abs(base[t])) * R.UB * 1.01 @ np.abs(d[t]) / step + 1e-6
            assert abs(float(dw[t, j]) - num) <= err
            y2 = y.copy()
            y2[rows[t, j], 5] += step
            up = loss(y2, w)
            num = ((up - base) * d).sum() / step
            err = (abs(up[t, 5]) + abs(base[t, 5])) * R.UB * 1.01 * abs(d[t, 5]) / step + R.UB * abs(num) * 2 + 1e-6
            assert abs(float(dy[rows[t, j], 5]) - num) <= err


def test_rows_outside_the_capacity_are_skipped():
    x = torch.ones((2, 16), dtype=torch.bfloat16, device="cuda:0")
    rows = torch.tensor([[0, 128], [-5, 1 << 30]], dtype=torch.int32, device="cuda:0")
    src = torch.full((128,), -1, dtype=torch.int32, device="cuda:0")
    src[0] = 0
    offs = torch.tensor([256], dtype=torch.int32, device="cuda:0")
    out = Guarded(2 * 128 * 16, torch.bfloat16, (128, 16))
    moe.moe_dispatch(x, rows, src, offs, out.t)
    c = torch.empty((2, 16), dtype=torch.bfloat16, device="cuda:0")
    moe.moe_combine(out.t, rows, c)
    torch.cuda.synchronize()
    assert out.guards_intact()
    assert float(out.t[0].sum()) == 16 and float(out.t[1:].abs().sum()) == 0
    assert float(c[0].sum()) == 16 and float(c[1].abs().sum()) == 0


def test_offsets_past_32_bits():
    """Packed buffers above 4 GiB: the last rows are written and read."""
    H = 8192
    cap = (1 << 32) // (2 * H) + 256
    T = 3
    rows = torch.tensor([[0], [cap - 129], [cap - 128]], dtype=torch.int32, device="cuda:0")
    src = torch.full((cap,), 0, dtype=torch.int32, device="cuda:0")     # no padding but the rows below
    src[cap - 127:] = -1
    offs = torch.tensor([cap], dtype=torch.int32, device="cuda:0")
    x = torch.randn((T, H), device="cuda:0").to(torch.bfloat16)
    out = torch.full((cap, H), 7.0, dtype=torch.bfloat16, device="cuda:0")
    moe.moe_dispatch(x, rows, src, offs, out)
    back = torch.empty_like(x)
    moe.moe_combine(out, rows, back)
    torch.cuda.synchronize()
    assert torch.equal(back, x)
    for t, r in enumerate((0, cap - 129, cap - 128)):
        assert torch.equal(out[r], x[t])
    assert float(out[cap - 127:].abs().sum()) == 0 and float(out[1]. sum()) == 7.0 * H


def test_another_stream():
    """The calls run on the stream they are given, in its order."""
    s = torch.cuda.Stream()
    T, H = 512, 1024
    x = torch.randn((T, H), device="cuda:0").to(torch.bfloat16)
    rows = torch.arange(T, dtype=torch.int32, device="cuda:0").view(T, 1)
    src = torch.arange(T, dtype=torch.int32, device="cuda:0")
    offs = torch.tensor([T], dtype=torch.int32, device="cuda:0")
    out, back = torch.zeros_like(x), torch.zeros_like(x)
    torch.cuda.synchronize()
    moe.moe_dispatch(x, rows, src, offs, out, stream=s)
    moe.moe_combine(out, rows, back, stream=s)
    s.synchronize()
    assert torch.equal(back, x)


def test_gradient_of_more_than_2_to_24_work_groups():
    """The most tokens there may be, one choice each, and as many rows."""
    T, H = moe.MAX_PAIRS, 16
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda:0")
    y = torch.full((T, H), 0.5, dtype=torch.bfloat16, device="cuda:0")
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda:0").view(T, 1)   # in reverse
    rows[T - 7] = -1                                                                     # row 6 is padding
    src = (T - 1 - torch.arange(T, dtype=torch.int32, device="cuda:0")).contiguous()
    src[6] = -1
    x[T - 1] = 3.0
    offs = torch.tensor([T], dtype=torch.int32, device="cuda:0")
    w = torch.full((T, 1), 2.0, device="cuda:0")
    out = torch.full((T, H), 9.0, dtype=torch.bfloat16, device="cuda:0")
    dw = torch.full((T, 1), 9.0, device="cuda:0")
    moe.moe_dispatch(x, rows, src, offs, out, weights=w, y=y, dweights=dw)
    torch.cuda.synchronize()
    want = torch.full((T, H), 2.0, dtype=torch.bfloat16, device="cuda:0")
    want[0], want[6] = 6.0, 0.0
    assert torch.equal(out, want)
    want = torch.full((T, 1), 8.0, device="cuda:0")
    want[T - 1], want[T - 7] = 24.0, 0.0
    assert torch.equal(dw, want)


def test_combine_of_more_than_2_to_24_work_groups():
    """2^24 tokens of four pieces each: 51 GB of output, most of it zeros."""
    T, H, cap = moe.MAX_PAIRS, 1552, 128
    y = torch.randn((cap, H), device="cuda:0").to(torch.bfloat16)
    rows = torch.full((T, 1), -1, dtype=torch.int32, device="cuda:0")
    some = [0, 1, T // 2, T - 2, T - 1]
    rows[some, 0] = torch.tensor([5, 0, 127, 64, 3], dtype=torch.int32, device="cuda:0")
    out = torch.full((T, H), 9.0, dtype=torch.bfloat16, device="cuda:0")
    moe.moe_combine(y, rows, out)
    torch.cuda.synchronize()
    assert torch.equal(out[some], y[[5, 0, 127, 64, 3]])
    out[some] = 0
    for part in out.split(1 << 20):
        assert not part.any()
