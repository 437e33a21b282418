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
