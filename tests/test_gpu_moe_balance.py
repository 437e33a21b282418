"""Balance loss of the router and its gradient on the GPU, against the plain
64-bit implementation and against differences."""
import numpy as np
import pytest
import torch

import i8_reference as I
import moe_reference as R
from gpu_helpers import Guarded, log
from nvfp4_block_scaled_group_amd import moe

pytestmark = pytest.mark.gpu

SCORES = {"softmax": moe.SCORE_SOFTMAX, "sigmoid": moe.SCORE_SIGMOID}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(seed, T, E, k, dtype):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)
    if T > 4:
        l[1] = -np.inf                                  # a token without experts
        l[2] = np.nan
        l[3, : E // 2] = -np.inf
        l[4, E - 1] = np.inf                            # counts as the largest finite value
        if E > 1:
            l[4, 0] = -3e38
    lt = torch.from_numpy(l.astype(np.float32)).to(TYPES[dtype])
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)       # some are no choice
    return rng, lt, lt.double().numpy(), ids


def buffers(T, E, S):
    ws = torch.full((moe.moe_balance_workspace(T, E, S),), 0xFF, dtype=torch.uint8, device="cuda:0")
    return dict(loss=Guarded(4, torch.float32), counts=Guarded(4 * S * E, torch.int32, (S, E)),
                probs=Guarded(4 * S * E, torch.float32, (S, E)), seq_tokens=Guarded(4 * S, torch.int32)), ws


def both(lt, ids, ends, score, coef, k, dloss=None, add=None, in_place=False):
    T, E = lt.shape
    S = 1 if ends is None else len(ends)
    out, ws = buffers(T, E, S)
    dev_l, e = lt.to("cuda:0"), None if ends is None else R.to_dev(np.asarray(ends, np.int32))
    how = dict(seq_ends=e, score=SCORES[score], coef=coef)
    t = {key: g.t for key, g in out.items()}
    moe.moe_balance(dev_l, R.to_dev(ids), **t, workspace=ws, **how)
    d = Guarded(T * E * lt.element_size(), lt.dtype, (T, E))
    if in_place:
        d.t.copy_(add)
        add = d.t
    moe.moe_balance_bwd(dev_l, t["counts"], t["seq_tokens"], d.t, topk=k, dloss=dloss, add=add, **how)
    torch.cuda.synchronize()
    assert d.guards_intact() and all(g.guards_intact() for g in out.values())
    return t, d.t


def rel_of(l, E):
    """Relative error of a probability: the exponent's argument is rounded (|l - max| of a few u), the hardware's
    exponential and reciprocal add a few u, and the sum over the experts at most one u a term."""
    fin = np.where(np.isfinite(l), l, 0.0)
    span = np.minimum(fin.max(1, keepdims=True) - fin, 120.0)          # beyond that it is 0 in fp32 too
    return (4 * np.maximum(span, np.minimum(np.abs(fin), 120.0)) + E + 24) * R.U


CASES = [  # T, E, k, ends
    (1, 1, 1, None), (1, 8, 2, None), (2, 33, 3, [1, 2]), (7, 2, 1, [0, 3, 3, 6]), (33, 8, 2, None), (128, 64, 6, None),
    (129, 64, 6, None), (130, 7, 3, [130]), (300, 100, 8, [5, 5, 140, 256, 290]), (700, 128, 4, [700]), (513, 200, 10, [128, 256, 384, 513]),
    (1000, 256, 8, None), (260, 512, 2, [100, 230]), (90, 700, 3, [40, 90]), (70, 1024, 16, None), (150, 2048, 5, [10, 149]),
    (140, 4096, 4, None), (40000, 16, 2, None), (33000, 40, 4, [1, 20000, 20001, 32000]), (257, 31, 2, list(range(1, 251))),
]


@pytest.mark.parametrize("T,E,k,ends", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_balance(T, E, k, ends, score, dtype):
    log(f"balance T={T} E={E} k={k} {score} {dtype}")
    rng, lt, l, ids = make(T + E, T, E, k, dtype)
    dloss = torch.tensor([1.5], device="cuda:0")
    add = torch.from_numpy((rng.standard_normal((T, E)) * 1e-3 / T).astype(np.float32)).to(lt.dtype)
    got, d = both(lt, ids, ends, score, 0.3, k, dloss, add.to("cuda:0"), in_place=T % 2 == 1)
    loss, counts, probs, tokens, grad, scale = I.balance(l, ids, ends, score, 0.3, k)
    assert np.array_equal(got["counts"].cpu().numpy(), counts)
    assert np.array_equal(got["seq_tokens"].cpu().numpy(), tokens)
    rel = rel_of(l, E)
    worst = float(rel.max())
    n = tokens[:, None].astype(np.float64)
    R.check(got["probs"], probs, probs * (worst + (n + 24) * R.U) + n * 1e-37, "probs")
    R.check(got["loss"], np.array([loss]), np.array([loss * (worst + (n.max() + E + len(tokens) + 40) * R.U) + 1e-37]), "loss")
    want = 1.5 * grad + add.double().numpy()
    # p, 1 - s and the inner sum each off by rel, and the factors' roundings
    err = 1.5 * scale * (3 * rel + worst + (E + 24) * R.U) + 2 * R.U * np.abs(want) + 1e-36
    if lt.dtype == torch.bfloat16:
        err = err + R.UB * (np.abs(want) + err)
    R.check(d, want, err, "dlogits")
    plain = torch.isnan(lt) | (lt == -float("inf"))
    assert torch.equal(d.cpu()[plain], add[plain])                     # masked: what was there before, exactly


@pytest.mark.parametrize("T,E,k,ends", [
    (70000, 3, 2, list(range(1, moe.MAX_SEQS)) + [69999]), (1 << 20, 16, 16, None), (1 << 20, 16, 16, [5, 5, 700000])])
def test_most_sequences_and_most_pairs(T, E, k, ends):
    log(f"balance T={T} E={E} k={k}")
    rng, lt, l, ids = make(T, T, E, k, "f32")
    got, d = both(lt, ids, ends, "softmax", 0.3, k)
    loss, counts, probs, tokens, grad, scale = I.balance(l, ids, ends, "softmax", 0.3, k)
    assert np.array_equal(got["counts"].cpu().numpy(), counts) and np.array_equal(got["seq_tokens"].cpu().numpy(), tokens)
    rel, n = rel_of(l, E), tokens[:, None].astype(np.float64)
    worst = float(rel.max())
    R.check(got["probs"], probs, probs * (worst + (n + 24) * R.U) + n * 1e-37, "probs")
    R.check(got["loss"], np.array([loss]), np.array([loss * (worst + (n.max() + E + len(tokens) + 40) * R.U) + 1e-37]), "loss")
    R.check(d, grad, scale * (3 * rel + worst + (E + 24) * R.U) + 2 * R.U * np.abs(grad) + 1e-36, "dlogits")


def test_without_options():
    rng, lt, l, ids = make(9, 50, 24, 3, "f32")
    _, d = both(lt, ids, None, "softmax", 1.0, 3)
    _, _, _, _, grad, scale = I.balance(l, ids, None, "softmax", 1.0, 3)
    R.check(d, grad, scale * (4 * rel_of(l, 24) + 60 * R.U) + 1e-36, "dlogits")
    assert (d.cpu()[torch.isnan(lt) | (lt == -float("inf"))] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_follows_differences(score):
    rng, lt, l, ids = make(21, 40, 12, 2, "f32")
    l = np.where(np.isposinf(l) | (np.abs(l) > 1e30), 3.0, l)
    lt = torch.from_numpy(l.astype(np.float32))
    l, ends = lt.double().numpy(), [17, 39]
    _, d = both(lt, ids, ends, score, 0.9, 2)
    num, eps = np.zeros_like(l), 1e-5
    for t in range(40):
        for e in range(12):
            if np.isfinite(l[t, e]):
                a, b = l.copy(), l.copy()
                a[t, e] += eps
                b[t, e] -= eps
                num[t, e] = (I.balance(a, ids, ends, score, 0.9, 2)[0] - I.balance(b, ids, ends, score, 0.9, 2)[0]) / (2 * eps)
    # eps^2 times a third derivative below the loss, and the cancellation of two losses near 1 in 64 bits
    assert np.abs(d.double().cpu().numpy() - num).max() < 1e-7


def test_no_tokens():
    out, ws = buffers(0, 24, 1)
    empty = torch.empty((0, 24), device="cuda:0")
    moe.moe_balance(empty, torch.empty((0, 2), dtype=torch.int32, device="cuda:0"), **{k: g.t for k, g in out.items()}, workspace=ws)
    assert float(out["loss"].t) == 0 and int(out["seq_tokens"].t) == 0
    assert not out["counts"].t.any() and not out["probs"].t.any()
    moe.moe_balance_bwd(empty, out["counts"].t, out["seq_tokens"].t, empty, topk=2)
    for ends in ([0, 0, 0], [0]):
        out, ws = buffers(5, 24, len(ends))
        l = torch.randn((5, 24), device="cuda:0")
        e = R.to_dev(np.asarray(ends, np.int32))
        t = {k: g.t for k, g in out.items()}
        moe.moe_balance(l, torch.zeros((5, 2), dtype=torch.int32, device="cuda:0"), **t, workspace=ws, seq_ends=e)
        d = torch.full((5, 24), 7.0, device="cuda:0")
        moe.moe_balance_bwd(l, t["counts"], t["seq_tokens"], d, topk=2, seq_ends=e)
        assert float(t["loss"]) == 0 and not t["counts"].any() and not d.any()


@pytest.mark.parametrize("T", [100, 1000])
def test_bad_ends_give_a_loss_that_is_no_number(T):
    rng, lt, _, ids = make(6, T, 16, 2, "f32")
    for ends in ([-5, T], [60, 30, T], [50, T + 1], [T, 10], [-1], [T + 7], [2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]):
        got, d = both(lt, ids, ends, "softmax", 1.0, 2)            # the guards around every output are checked inside
        assert torch.isnan(got["loss"]).all(), ends


def test_counts_of_ranks_may_be_summed():
    """Two halves with summed counts give the gradient of the whole batch."""
    rng, lt, l, ids = make(30, 400, 32, 4, "f32")
    whole, d = both(lt, ids, None, "sigmoid", 0.5, 4)
    parts = [both(lt[i:i + 200], ids[i:i + 200], None, "sigmoid", 0.5, 4)[0] for i in (0, 200)]
    counts, tokens = parts[0]["counts"] + parts[1]["counts"], parts[0]["seq_tokens"] + parts[1]["seq_tokens"]
    assert torch.equal(counts, whole["counts"]) and torch.equal(tokens, whole["seq_tokens"])
    for i in (0, 200):
        half = torch.empty((200, 32), device="cuda:0")
        moe.moe_balance_bwd(lt[i:i + 200].to("cuda:0"), counts, tokens, half, topk=4, score=moe.SCORE_SIGMOID, coef=0.5)
        assert torch.equal(half, d[i:i + 200])


def test_rows_that_start_between_alignments():
    """Logits and gradients that are views four bytes into a buffer."""
    rng, lt, l, ids = make(12, 65, 64, 2, "f32")
    base = torch.zeros(65 * 64 + 1, device="cuda:0")
    view = base[1:].view(65, 64)
    view.copy_(lt)
    want, dwant = both(lt, ids, None, "softmax", 1.0, 2)
    out, ws = buffers(65, 64, 1)
    t = {k: g.t for k, g in out.items()}
    moe.moe_balance(view, R.to_dev(ids), **t, workspace=ws)
    dbase = torch.zeros(65 * 64 + 1, device="cuda:0")
    moe.moe_balance_bwd(view, t["counts"], t["seq_tokens"], dbase[1:].view(65, 64), topk=2)
    for key in t:
        assert torch.equal(t[key], want[key]), key
    assert torch.equal(dbase[1:].view(65, 64), dwant) and float(dbase[0]) == 0


def test_results_do_not_depend_on_the_run_and_replay():
    """Several runs, and replays of a captured graph with new logits, against the eager call's bits."""
    T, E, k, ends = 3000, 64, 6, [900, 901, 2900]
    rng, lt, _, ids = make(14, T, E, k, "bf16")
    first, dfirst = both(lt, ids, ends, "softmax", 0.1, k)
    for _ in range(3):
        again, d = both(lt, ids, ends, "softmax", 0.1, k)
        assert torch.equal(d, dfirst) and all(torch.equal(again[key], first[key]) for key in first)
    l, dev_ids, e = lt.to("cuda:0"), R.to_dev(ids), R.to_dev(np.asarray(ends, np.int32))
    b, dl = moe.alloc_balance(T, E, 3), torch.empty_like(l)

    def step():
        moe.moe_balance(l, dev_ids, **b, seq_ends=e, coef=0.1)
        moe.moe_balance_bwd(l, b["counts"], b["seq_tokens"], dl, topk=k, seq_ends=e, coef=0.1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        lt2 = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(torch.bfloat16)
        want, dwant = both(lt2, ids, ends, "softmax", 0.1, k)
        l.copy_(lt2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dl, dwant), i
        assert all(torch.equal(b[key], want[key]) for key in want), i


def least_us(call, reps=9):
    times = []
    for _ in range(reps):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


@pytest.mark.parametrize("where", ["behind", "between"])
def test_long_runs_of_empty_sequences(where):
    """Ends padded to a fixed number, the usual form for captured graphs: the real sequences get the same bits, the
    empty ones nothing, and the call takes about as long as one whose sequences are all empty (one after another the
    empty ones took five times as long)."""
    T, E, k, S = 8191, 64, 6, moe.MAX_SEQS
    rng, lt, l, ids = make(17, T, E, k, "f32")
    real = [0, 700, 1500, 1500, 4000, 5000, 8000]                    # rows behind the last one: padding
    cut = len(real) if where == "behind" else 3                      # real sequences before the long run
    ends = real[:cut] + [real[cut - 1]] * (S - len(real)) + real[cut:]
    log(f"balance {S} sequences, empty ones {where}")
    got, d = both(lt, ids, ends, "softmax", 0.3, k)
    few, dfew = both(lt, ids, real, "softmax", 0.3, k)
    at = torch.tensor([i for i in range(S) if i < cut or i >= S - len(real) + cut], device="cuda:0")
    for key in ("counts", "probs", "seq_tokens"):
        assert torch.equal(got[key][at], few[key]), key
        assert int((got[key] != 0).sum()) == int((few[key] != 0).sum()), key
    # the mean is over all sequences: the same sum over another number (a weight has five roundings), in other parts
    assert abs(float(got["loss"]) * S / len(real) - float(few["loss"])) < 64 * R.U * float(few["loss"])
    assert float((d.double() * (S / len(real)) - dfew.double()).abs().max()) < 16 * R.U * float(dfew.abs().max())
    dev_l, dev_ids, b = lt.to("cuda:0"), R.to_dev(ids), moe.alloc_balance(T, E, S)

    def call(e):
        e = R.to_dev(np.asarray(e, np.int32))
        return least_us(lambda: moe.moe_balance(dev_l, dev_ids, **b, seq_ends=e))

    padded, empty = call(ends), call([0] * S)
    log(f"padded {padded:.0f} us, all empty {empty:.0f} us")
    assert padded < 2 * empty


def test_the_most_sequences_do_not_wait_for_each_other():
    """65535 joining work-groups: 0.24 ms; 1.15 ms where each of them counts itself before the next can."""
    T, E, S = 64, 8, moe.MAX_SEQS
    b = moe.alloc_balance(T, E, S)
    l, ids = torch.randn((T, E), device="cuda:0"), torch.zeros((T, 1), dtype=torch.int32, device="cuda:0")
    e = torch.zeros(S, dtype=torch.int32, device="cuda:0")
    us = least_us(lambda: moe.moe_balance(l, ids, **b, seq_ends=e))
    log(f"{S} empty sequences {us:.0f} us")
    assert us < 600


@pytest.mark.parametrize("S,E", [(4, 1024), (5, 1024), (128, 30), (129, 30)])
def test_sequences_are_added_by_the_last_one_or_apart(S, E):
    """128 and more joining work-groups (32 experts of a sequence each), several calls on one workspace, replays."""
    T, k = 700, 3
    rng, lt, l, ids = make(S, T, E, k, "f32")
    ends = np.sort(rng.integers(0, T + 1, S)).astype(np.int32)
    first, d = both(lt, ids, ends, "softmax", 0.3, k)
    loss = I.balance(l, ids, ends, "softmax", 0.3, k)[0]
    # a lane adds at most 32 rows, the waves 16, the join 256 slots of 32 parts, 32 columns and the shares in order
    assert abs(float(first["loss"]) - loss) < (float(rel_of(l, E).max()) + 256 * R.U) * loss
    dev_l, dev_ids, e, b = lt.to("cuda:0"), R.to_dev(ids), R.to_dev(ends), moe.alloc_balance(T, E, S)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_balance(dev_l, dev_ids, **b, seq_ends=e, coef=0.3)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_balance(dev_l, dev_ids, **b, seq_ends=e, coef=0.3)
    for i in range(4):
        b["loss"].fill_(7)
        g.replay() if i % 2 else moe.moe_balance(dev_l, dev_ids, **b, seq_ends=e, coef=0.3)
        torch.cuda.synchronize()
        assert all(torch.equal(b[key], first[key]) for key in first), i


SUMS = [  # T, E, k, ends: all chunks and slots in use, one work-group alone, as many sequences as there can be
    (1 << 20, 16, 16, None), (1 << 20, 16, 16, [5, 5, 700000]), (40000, 16, 2, None), (33000, 40, 4, [1, 20000, 20001, 32000]),
    (1000, 256, 8, None), (128, 64, 6, None), (140, 4096, 4, None), (300, 2048, 5, [10, 290]),
    (70000, 3, 2, list(range(1, moe.MAX_SEQS)) + [69999]), (70000, 64, 2, list(range(1, moe.MAX_SEQS)) + [69999]),
]


@pytest.mark.parametrize("at", range(len(SUMS)))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_are_off_by_their_depth(at, score):
    """Bounds that the rows of a fraction of a chunk would pass, if they were lost (test_i8_host.py shows it)."""
    T, E, k, ends = SUMS[at]
    log(f"balance sums T={T} E={E} k={k} {score}")
    rng, lt, l, ids = make(T + E + 1, T, E, k, "f32")
    got, _ = both(lt, ids, ends, score, 0.3, k)
    loss, counts, probs, tokens, _, _ = I.balance(l, ids, ends, score, 0.3, k)
    off, loss_off = I.balance_bounds(l, ids, ends, score, 0.3, k, rel_of(l, E))
    R.check(got["probs"], probs, off, "probs")
    R.check(got["loss"], np.array([loss]), np.array([loss_off]), "loss")
