"""The 8-bit operators together, as ``examples/moe_layer_8bit.py`` runs them: a
training step with the balance loss and the 8-bit checkpoint, and serving with
8-bit integer weights, against the same layer in plain torch fp32 without any
cast; captured in graphs; on other streams and two at once."""
import os
import sys
import threading

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
sys.path.insert(0, os.path.join(ROOT, "tests"))

from test_gpu_moe_layer import E, F, H, K, T, off, plain, rand, rel, replays  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def made():
    import moe_layer_8bit as L
    g = torch.Generator(device="cuda:0")
    g.manual_seed(5)
    w = (rand(g, E, 2 * F, H, scale=H ** -0.5), rand(g, E, H, F, scale=F ** -0.5), rand(g, E, H, scale=H ** -0.5))
    shared = rand(g, H, H, scale=H ** -0.5)
    return L, g, w, shared, L.KeptLayer(*w, K, coef=0.3), L.Int8Layer(*w, shared, K)


def balance(logits, ids, ends, coef):
    """The loss with autograd, counts held constant."""
    p, loss, b = torch.softmax(logits, 1), 0.0, 0
    for e in ends:
        n = e - b
        counts = torch.bincount(ids[b:e].reshape(-1).long(), minlength=E).double()
        loss = loss + coef / len(ends) * E / (K * n * n) * (counts * p[b:e].double().sum(0)).sum()
        b = e
    return loss


def test_training_step(made):
    L, g, w, _, layer, _ = made
    x, dy = rand(g, T, H), rand(g, T, H)
    ends = [100, 110, T]
    d_ends = torch.tensor(ends, dtype=torch.int32, device="cuda:0")
    dloss = torch.tensor([40.0], device="cuda:0")
    y, loss, kept = layer.forward(x, d_ends)
    dx, dlogits, d_gu, d_down = layer.backward(dy, kept, dloss)
    assert int(kept["plan"]["d_status"]) == 0
    leaves = [t.float().requires_grad_() for t in (x, w[0], w[1])]
    logits = kept["logits"].clone().requires_grad_()
    top = torch.topk(logits, K, dim=1)
    assert torch.equal(top.indices.int(), kept["ids"])
    want = plain(leaves[0], (leaves[1], leaves[2], w[2]), kept["ids"], torch.softmax(top.values, 1))
    want.backward(dy.float(), retain_graph=True)
    through_weights = logits.grad.clone()
    # the checkpoint adds under 1% (its step is a 127th of a group's largest) to what the casts are off by
    assert rel(y, want) < off(6)
    assert rel(d_down, leaves[2].grad) < off(6) + 0.01
    assert rel(d_gu, leaves[1].grad) < off(8) + 0.01
    assert rel(dx, leaves[0].grad) < off(8) + 0.01
    # the balance loss reads the logits as they are: fp32 alone
    logits.grad = None
    ref = balance(logits, kept["ids"], ends, layer.coef)
    ref.backward()
    assert abs(float(loss) - float(ref)) < 1e-5 * float(ref)
    assert rel(dlogits, through_weights + 40.0 * logits.grad) < off(6)
    only = torch.empty_like(dlogits)
    L.moe.moe_balance_bwd(kept["logits"], kept["balance"]["counts"], kept["balance"]["seq_tokens"], only, topk=K,
                          seq_ends=d_ends, coef=layer.coef)
    assert rel(only, logits.grad) < 1e-5


# The cast of a line of n normal values to 8 bits has a step of amax / 127, and
# amax is below 4.5 of their sigma for any n here, so a code is off by at most
# 4.5 / 127 / sqrt(12) = 1.03% of sigma in the root mean square.  Casts are
# independent: n of them are off by sqrt(n) of that; bf16 roundings of results
# add 2^-9 each, far below.
def off8(n):
    return 0.0103 * n ** 0.5 + 0.004


def served(x, w, shared, layer):
    _, ids, weights = layer.route(x)
    return plain(x, w, ids, weights) + x.float() @ shared.float().t()


def test_serving_a_batch_and_tokens(made):
    L, g, w, shared, _, layer = made
    x = rand(g, T, H)
    want = served(x, w, shared, layer)
    assert rel(layer.batch(x), want) < off8(6)             # x three times, the weights of gate and up, hidden and down
    for n in (1, 7, 40):
        few = x[:n].contiguous()
        y = layer.decode(few)
        assert rel(y, want[:n]) < off8(6)
        # both forms make the same codes; hidden rows and results differ in the roundings to bf16 alone
        assert rel(layer.batch(few), y) < 0.01
        assert rel(layer.project(few), few.float() @ shared.float().t()) < off8(2)


def test_training_calls_replay_in_a_graph(made):
    """Balance loss, block with checkpoint and their gradients under routing that changes between the replays."""
    L, g, w, _, layer, _ = made
    m, dev = L.moe, "cuda:0"
    plan, bal = m.alloc_plan(T, K, E), m.alloc_balance(T, E, 3)
    cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]

    def b16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=dev)

    logits, ids, wt = torch.empty((T, E), device=dev), torch.zeros((T, K), dtype=torch.int32, device=dev), torch.zeros((T, K), device=dev)
    ends = torch.zeros(3, dtype=torch.int32, device=dev)
    x, packed, hid, again, dgu = b16(T, H), b16(cap, H), b16(cap, F), b16(cap, F), b16(cap, 2 * F)
    dw, dlogits, kept = torch.zeros((T, K), device=dev), torch.zeros((T, E), device=dev), m.alloc_keep8(cap, F)
    cast = L.B.alloc_outputs(cap, H, E, True, False, device=dev)
    kept["gu8"].zero_()
    kept["gu_scale"].zero_()

    def step():
        m.moe_route(logits, ids, wt)
        m.moe_balance(logits, ids, **bal, seq_ends=ends, coef=0.1)
        m.moe_plan(ids, **plan)
        m.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        L.B.nvfp4_group_quantize_graphsafe(packed, E, offs, status, **cast)
        rows = cast["row_data"], cast["row_scale"], cast["row_amax"]
        m.moe_glu_keep8_graphsafe(*rows, *layer.gu_lines, offs, hid, **kept, d_status=status)
        m.moe_glu_bwd_keep8_graphsafe(*rows, *layer.down_turned, offs, **kept, dgu=dgu, d_status=status, h=again)
        m.moe_route_bwd(logits, ids, wt, dlogits)
        m.moe_balance_bwd(logits, bal["counts"], bal["seq_tokens"], dlogits, topk=K, seq_ends=ends, coef=0.1, add=dlogits)

    def refresh():
        x.copy_(rand(g, T, H))
        logits.copy_(x.float() @ layer.router.t() + 2 * torch.randn(E, generator=g, device=dev))
        ends.copy_(torch.sort(torch.randint(0, T + 1, (3,), generator=g, device=dev)).values)

    refresh()
    replays(step, refresh, [hid, again, dgu, dlogits, kept["gu8"], kept["gu_scale"], bal["loss"], bal["counts"], bal["probs"],
                            bal["seq_tokens"]])
    assert int(status) == 0


def test_serving_replays_in_a_graph(made):
    """The packed form under changing routing, the token form and the projection in each of its sizes."""
    L, g, w, shared, _, layer = made
    m, i8, dev = L.moe, L.i8, "cuda:0"
    plan = m.alloc_plan(T, K, E)
    cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
    ids, wt, logits = torch.zeros((T, K), dtype=torch.int32, device=dev), torch.zeros((T, K), device=dev), torch.empty((T, E), device=dev)
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    packed, hid = (torch.zeros((cap, n), dtype=torch.bfloat16, device=dev) for n in (H, F))
    out, y = torch.zeros((cap, H), device=dev), torch.zeros((T, H), dtype=torch.bfloat16, device=dev)
    a, b = i8.alloc_cast(cap, H), i8.alloc_cast(cap, F)
    few = (1, 16, 40, T)
    ps = [torch.zeros((n, H), dtype=torch.bfloat16, device=dev) for n in few]
    ws = torch.empty(i8.i8_linear_workspace(T, H, H), dtype=torch.uint8, device=dev)
    th, ty = torch.zeros((5 * K, F), dtype=torch.bfloat16, device=dev), torch.zeros((5 * K, H), device=dev)
    c = i8.alloc_cast(T, H)

    def step():
        m.moe_route(logits, ids, wt)
        m.moe_plan(ids, **plan)
        m.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        i8.i8_group_cast_graphsafe(packed, offs, **a, d_status=status)
        i8.i8_group_glu_graphsafe(*a.values(), *layer.gate_up, offs, hid, status)
        i8.i8_group_cast_graphsafe(hid, offs, **b, d_status=status)
        i8.i8_group_gemm_graphsafe(*b.values(), *layer.down, offs, out, status)
        m.moe_combine(out, plan["rows"], y, weights=wt)
        i8.i8_group_cast(x, **c)
        for n, p in zip(few, ps):                                   # one workspace, call after call
            i8.i8_linear(c["q"][:n], c["scale"][:n], *layer.shared, p, ws)
        i8.i8_token_glu(x[:5], ids[:5], *layer.gate_up, th)
        i8.i8_token_linear(th, ids[:5], *layer.down, ty)

    def refresh():
        x.copy_(rand(g, T, H))
        logits.copy_(x.float() @ layer.router.t() + 2 * torch.randn(E, generator=g, device=dev))

    refresh()
    replays(step, refresh, [hid, out, y, th, ty, *ps])
    assert int(status) == 0


def test_other_streams_and_two_calls_at_once(made):
    """Two host threads on streams of their own, with buffers of their own: each the bits of the call alone."""
    L, g, w, shared, kept_layer, layer = made
    xs = [rand(g, T, H) for _ in range(2)]
    alone = [(layer.batch(x), layer.decode(x[:5].contiguous()), *kept_layer.forward(x)[:2]) for x in xs]
    torch.cuda.synchronize()
    errors = []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = (layer.batch(xs[i]), layer.decode(xs[i][:5].contiguous()), *kept_layer.forward(xs[i])[:2])
                    s.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, alone[i]))
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors


def test_examples_run(capsys, monkeypatch):
    import moe_layer_8bit as L
    monkeypatch.setattr(sys, "argv", ["moe_layer_8bit.py", "--tokens", "200", "--hidden", "256", "--inner", "128", "--experts", "8",
                                      "--topk", "2"])
    L.main()
    assert "balance loss" in capsys.readouterr().out


def test_two_calls_at_once_all_end(made):
    """As above, with a record of every round: a thread that stops short, or does not end, fails."""
    L, g, w, shared, kept_layer, layer = made
    xs = [rand(g, T, H) for _ in range(2)]
    alone = [(layer.batch(x), layer.decode(x[:5].contiguous()), *kept_layer.forward(x)[:2]) for x in xs]
    torch.cuda.synchronize()
    rounds, errors = [[], []], []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for n in range(10):
                    got = (layer.batch(xs[i]), layer.decode(xs[i][:5].contiguous()), *kept_layer.forward(xs[i])[:2])
                    s.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, alone[i])), n
                    rounds[i].append(n)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,), daemon=True) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors
    assert not any(t.is_alive() for t in threads) and rounds == [list(range(10))] * 2
