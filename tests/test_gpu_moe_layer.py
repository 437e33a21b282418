"""The operators together, as ``examples/moe_layer.py`` runs them: one expert
layer's forward and backward pass, its decoding form and the adapted input
projection, against the same layer in plain torch fp32 without any cast."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

T, H, F, E, K = 300, 256, 128, 8, 3


def rand(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda:0") * scale).to(torch.bfloat16)


@pytest.fixture(scope="module")
def made():
    import moe_layer as L
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)
    w = (rand(g, E, 2 * F, H, scale=H ** -0.5), rand(g, E, H, F, scale=F ** -0.5), rand(g, E, H, scale=H ** -0.5))
    return L, g, w, L.ExpertLayer(*w, K)


def plain(x, w, ids, weights):
    """The layer in fp32, choices given."""
    gu_w, down, _ = (t.float() for t in w)
    x = x.float()
    y = torch.zeros_like(x)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        g, u = (x[t] @ gu_w[e].t()).chunk(2, 1)
        y = y.index_add(0, t, weights[t, j][:, None] * ((g * torch.sigmoid(g) * u) @ down[e].t()))
    return y


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


# A cast to E2M1 with block scales is off by about 10% of a tensor of normal
# values in the 2-norm (the grid's gaps are a third to a half of the smaller
# neighbour, the block's largest sits at 6); 0.11 leaves room for the scale's
# own rounding.  The casts are independent, so a result that n cast operands
# enter is off by sqrt(n) of that.
def off(n):
    return 0.11 * n ** 0.5


def test_forward_and_backward(made):
    L, g, w, layer = made
    x, dy = rand(g, T, H), rand(g, T, H)
    y, kept = layer.forward(x)
    dx, dlogits, d_gu, d_down = layer.backward(dy, kept)
    assert int(kept["plan"]["d_status"]) == 0
    leaves = [t.float().requires_grad_() for t in (x, w[0], w[1])]
    logits = (x.float() @ w[2].float().t()).requires_grad_()
    top = torch.topk(logits, K, dim=1)
    assert torch.equal(top.indices.int(), kept["ids"])
    want = plain(leaves[0], (leaves[1], leaves[2], w[2]), kept["ids"], torch.softmax(top.values, 1))
    want.backward(dy.float())
    assert rel(y, want) < off(6)           # x and weights of gate and of up, the hidden rows, down
    assert rel(d_down, leaves[2].grad) < off(6)      # dy, the hidden rows and what made them
    assert rel(dlogits, logits.grad) < off(6)        # the forward pass's rows
    assert rel(d_gu, leaves[1].grad) < off(8)        # dy and down, x and weights of gate and of up, dgu, x
    assert rel(dx, leaves[0].grad) < off(8)


def test_decode_agrees_with_the_batch_and_with_plain(made):
    L, g, w, layer = made
    x = rand(g, 7, H)
    y = layer.decode(x)
    _, ids, weights = layer.route(x)
    want = plain(x, w, ids, weights)
    assert rel(y, want) < off(3)           # the weights of gate, up and down
    assert rel(layer.forward(x)[0], y) < off(3)   # x twice, the hidden rows


def test_projection_with_adapters(made):
    L, g, w, _ = made
    p, a, b = rand(g, H, H, scale=H ** -0.5), rand(g, 4, 16, H, scale=H ** -0.5), rand(g, 4, H, 16, scale=0.25)
    alpha = torch.tensor([1.0, 0.5, 2.0, -1.0], device="cuda:0")
    x, ids = rand(g, 9, H), torch.tensor([3, -1, 0, 0, 2, 1, -1, 3, 2], dtype=torch.int32, device="cuda:0")
    y = L.AdaptedProjection(p, a, b, alpha)(x, ids)
    want = x.float() @ p.float().t()
    for t, i in enumerate(ids.tolist()):
        if i >= 0:
            want[t] += alpha[i] * (b[i].float() @ (a[i].float() @ x[t].float()))
    assert rel(y, want) < off(1)


def test_a_decoding_step_replays_in_a_graph(made):
    """Captured once, replayed on new tokens with eager work between."""
    L, g, w, layer = made
    x = rand(g, 5, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, wt = torch.empty((5, K), dtype=torch.int32, device="cuda:0"), torch.empty((5, K), device="cuda:0")
    logits = torch.empty((5, E), device="cuda:0")
    hid = torch.empty((5 * K, F), dtype=torch.bfloat16, device="cuda:0")
    out, y = torch.empty((5 * K, H), device="cuda:0"), torch.empty((5, H), dtype=torch.bfloat16, device="cuda:0")
    rows = torch.arange(5 * K, dtype=torch.int32, device="cuda:0").view(5, K)

    def step():
        L.moe.moe_route(logits, ids, wt)
        L.moe.moe_token_glu(x, ids, *layer.gu_lines, hid)
        L.moe.moe_token_linear(hid, ids, *layer.down_lines, out)
        L.moe.moe_combine(out, rows, y, weights=wt)

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        x.copy_(rand(g, 5, H))
        logits.copy_(x.float() @ layer.router.t())
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def replays(step, refresh, outputs):
    """Captures step, then replays it on new inputs with eager work between;
    every replay gives the eager call's bits."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        refresh()
        for t in outputs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs]
        for t in outputs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outputs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert any(t.any() for t in got)


def test_training_calls_replay_in_a_graph(made):
    """Plan, dispatch, block, its backward pass, combine and their gradients
    under a routing that changes between the replays."""
    L, g, w, layer = made
    m, dev = L.moe, "cuda:0"
    plan = m.alloc_plan(T, K, E)
    cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]

    def b16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=dev)

    logits, ids, wt = torch.empty((T, E), device=dev), torch.zeros((T, K), dtype=torch.int32, device=dev), torch.zeros((T, K), device=dev)
    x, packed, hid, gu, y = b16(T, H), b16(cap, H), b16(cap, F), b16(cap, 2 * F), b16(T, H)
    out = torch.zeros((cap, H), device=dev)
    d_out, dw, dlogits, dgu, dx = b16(cap, H), torch.zeros((T, K), device=dev), torch.zeros((T, E), device=dev), b16(cap, 2 * F), b16(T, H)
    cast = [L.B.alloc_outputs(cap, n, E, True, False, device=dev) for n in (H, F, H)]

    def rows(c, t):
        L.B.nvfp4_group_quantize_graphsafe(t, E, offs, status, **c)
        return c["row_data"], c["row_scale"], c["row_amax"]

    def step():
        m.moe_route(logits, ids, wt)
        m.moe_plan(ids, **plan)
        m.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        m.moe_glu_graphsafe(*rows(cast[0], packed), *layer.gu_lines, offs, hid, status, gu=gu)
        L.B.nvfp4_group_gemm_graphsafe(*rows(cast[1], hid), *layer.down_lines, offs, out, status)
        m.moe_combine(out, plan["rows"], y, weights=wt)
        m.moe_dispatch(x, plan["rows"], plan["src"], offs, d_out, weights=wt, y=out, dweights=dw)
        m.moe_route_bwd(logits, ids, dw, dlogits)
        m.moe_glu_bwd_graphsafe(*rows(cast[2], d_out), *layer.down_turned, offs, gu, dgu, status)
        m.moe_combine(d_out, plan["rows"], dx)

    def refresh():
        x.copy_(rand(g, T, H))
        logits.copy_(x.float() @ layer.router.t() + 2 * torch.randn(E, generator=g, device=dev))

    refresh()
    replays(step, refresh, [ids, wt, plan["rows"], plan["src"], plan["d_offs"], plan["counts"], packed, hid, gu, out, y, d_out, dw,
                            dlogits, dgu, dx])
    assert int(status) == 0


@pytest.mark.parametrize("rows,k", [(7, 256), (200, 256), (60, 2048)])
def test_adapted_projection_replays_in_a_graph(made, rows, k):
    L, g, _, _ = made
    n, r, a = 512, 16, 5
    p = L.AdaptedProjection(rand(g, n, k, scale=k ** -0.5), rand(g, a, r, k, scale=k ** -0.5), rand(g, a, n, r, scale=0.25),
                            torch.linspace(0.5, 2.0, a, device="cuda:0"))
    x, y = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda:0"), torch.empty((rows, n), dtype=torch.bfloat16, device="cuda:0")
    ids = torch.empty(rows, dtype=torch.int32, device="cuda:0")
    ws = torch.empty(L.moe.lora_workspace(rows, k, n, r), dtype=torch.uint8, device="cuda:0")

    def refresh():
        x.copy_(rand(g, rows, k))
        ids.copy_(torch.randint(-1, a, (rows,), generator=g, device="cuda:0"))

    refresh()
    replays(lambda: L.moe.lora_linear(x, *p.w, *p.lora, ids, p.alpha, y, ws), refresh, [y])
