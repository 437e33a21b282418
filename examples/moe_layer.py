"""One mixture-of-experts layer on the library's operators.

    python examples/moe_layer.py [--tokens 4096] [--hidden 2048] [--inner 1024] [--experts 32] [--topk 4]

``ExpertLayer`` keeps the experts' weights as row-scaled NVFP4 (cast once) and
runs

* ``forward`` / ``backward``: a training step's batch.  Route, plan, dispatch
  into packed 128-row groups, cast, gate and up projection with activation and
  product, cast, down projection, combine; and the gradients of the tokens,
  the router's logits and every expert weight;
* ``decode``: a few tokens of decoding requests against the same weights, with
  no packing and no activation cast;
* ``project``: the layer's input projection with a low-rank adapter for each
  request.

Everything is enqueued on the current stream; the routing stays on the device.
Run as a program it does one step of each and prints their times.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from nvfp4_block_scaled_group_amd import binding as B  # noqa: E402
from nvfp4_block_scaled_group_amd import moe  # noqa: E402


def cast_weights(w):
    """bf16 weights [E, n, k] -> their lines [E, n, k] and the lines of the transpose [E, k, n], both NVFP4
    (data, scale, amax).  n and k multiples of 128."""
    E, n, k = w.shape
    out = B.alloc_outputs(E * n, k, E, device=w.device)
    B.nvfp4_group_quantize(w.view(E * n, k), [n] * E, **out)
    lines = (out["row_data"].view(E, n, k // 2), out["row_scale"].view(E, n, k // 16), out["row_amax"])
    turned = (out["col_data"].view(E, k, n // 2), out["col_scale"].view(E, k, n // 16), out["col_amax"])
    return lines, turned


class ExpertLayer:
    """gate_up [E, 2f, h], down [E, h, f], router [E, h] in bf16."""

    def __init__(self, gate_up, down, router, topk):
        self.E, self.f2, self.h = gate_up.shape
        self.f, self.topk, self.router = self.f2 // 2, topk, router.float()
        self.gu_lines, self.gu_turned = cast_weights(gate_up)
        self.down_lines, self.down_turned = cast_weights(down)
        self.dev = gate_up.device

    def _quantize(self, x, plan):
        out = B.alloc_outputs(x.shape[0], x.shape[1], self.E, device=self.dev)
        B.nvfp4_group_quantize_graphsafe(x, self.E, plan["d_offs"], plan["d_status"], **out)
        rows = (out["row_data"], out["row_scale"], out["row_amax"])
        return rows, (out["col_data"], out["col_scale"], out["col_amax"])

    def _bf16(self, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=self.dev)

    def route(self, x):
        """Logits of the router and the chosen experts with their weights."""
        T = x.shape[0]
        logits = x.float() @ self.router.t()
        ids = torch.empty((T, self.topk), dtype=torch.int32, device=self.dev)
        weights = torch.empty((T, self.topk), device=self.dev)
        moe.moe_route(logits, ids, weights)
        return logits, ids, weights

    def forward(self, x):
        """x [T, h] bf16 -> y [T, h] bf16, and what backward needs."""
        T = x.shape[0]
        logits, ids, weights = self.route(x)
        plan = moe.alloc_plan(T, self.topk, self.E, device=self.dev)
        moe.moe_plan(ids, **plan)
        cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
        packed = self._bf16(cap, self.h)
        moe.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        x_rows, x_cols = self._quantize(packed, plan)
        hidden, gu = self._bf16(cap, self.f), self._bf16(cap, self.f2)
        moe.moe_glu_graphsafe(*x_rows, *self.gu_lines, offs, hidden, status, gu=gu)
        h_rows, h_cols = self._quantize(hidden, plan)
        out = torch.empty((cap, self.h), device=self.dev)
        B.nvfp4_group_gemm_graphsafe(*h_rows, *self.down_lines, offs, out, status)
        y = self._bf16(T, self.h)
        moe.moe_combine(out, plan["rows"], y, weights=weights)
        return y, dict(logits=logits, ids=ids, weights=weights, plan=plan, x_cols=x_cols, gu=gu, h_cols=h_cols, out=out)

    def backward(self, dy, kept):
        """dy [T, h] bf16 -> gradients of x (through the experts), the logits, gate_up and down."""
        T, plan = dy.shape[0], kept["plan"]
        cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
        # combine: gradient rows, scaled by the weights, and the weights' own gradient
        d_out, dw = self._bf16(cap, self.h), torch.empty((T, self.topk), device=self.dev)
        moe.moe_dispatch(dy, plan["rows"], plan["src"], offs, d_out, weights=kept["weights"], y=kept["out"], dweights=dw)
        dlogits = torch.empty_like(kept["logits"])
        moe.moe_route_bwd(kept["logits"], kept["ids"], dw, dlogits)
        # down projection and activation
        do_rows, do_cols = self._quantize(d_out, plan)
        dgu = self._bf16(cap, self.f2)
        moe.moe_glu_bwd_graphsafe(*do_rows, *self.down_turned, offs, kept["gu"], dgu, status)
        d_down = torch.empty((self.E, self.h, self.f), device=self.dev)
        B.nvfp4_group_gemm_wgrad_graphsafe(*do_cols, *kept["h_cols"], cap, self.E, offs, self.h, self.f, d_down, status)
        # gate and up projection
        dgu_rows, dgu_cols = self._quantize(dgu, plan)
        d_packed = torch.empty((cap, self.h), device=self.dev)
        B.nvfp4_group_gemm_graphsafe(*dgu_rows, *self.gu_turned, offs, d_packed, status)
        d_gu = torch.empty((self.E, self.f2, self.h), device=self.dev)
        B.nvfp4_group_gemm_wgrad_graphsafe(*dgu_cols, *kept["x_cols"], cap, self.E, offs, self.f2, self.h, d_gu, status)
        dx = self._bf16(T, self.h)
        moe.moe_combine(d_packed, plan["rows"], dx)
        return dx, dlogits, d_gu, d_down

    def decode(self, x):
        """x [T, h] bf16 of a few requests -> y [T, h] bf16 against the same weights."""
        T = x.shape[0]
        _, ids, weights = self.route(x)
        hidden = self._bf16(T * self.topk, self.f)
        moe.moe_token_glu(x, ids, *self.gu_lines, hidden)
        out = torch.empty((T * self.topk, self.h), device=self.dev)
        moe.moe_token_linear(hidden, ids, *self.down_lines, out)
        rows = torch.arange(T * self.topk, dtype=torch.int32, device=self.dev).view(T, self.topk)
        y = self._bf16(T, self.h)
        moe.moe_combine(out, rows, y, weights=weights)
        return y


class AdaptedProjection:
    """A projection [n, k] shared by all requests, with low-rank adapters lora_a [A, r, k], lora_b [A, n, r]."""

    def __init__(self, w, lora_a, lora_b, alpha):
        (data, scale, amax), _ = cast_weights(w[None])
        self.w, self.lora = (data[0], scale[0], amax), (lora_a, lora_b)
        self.alpha = alpha

    def __call__(self, x, adapter_ids):
        """x [T, k] bf16, adapter_ids [T] i32 (-1: none) -> [T, n] bf16."""
        T, k = x.shape
        n, r = self.w[0].shape[0], self.lora[0].shape[1]
        y = torch.empty((T, n), dtype=torch.bfloat16, device=x.device)
        ws = torch.empty(moe.lora_workspace(T, k, n, r), dtype=torch.uint8, device=x.device)
        moe.lora_linear(x, *self.w, *self.lora, adapter_ids, self.alpha, y, ws)
        return y


def timed(fn, reps=20):
    fn()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def arguments(doc):
    ap = argparse.ArgumentParser(description=doc, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    return ap.parse_args()


def generator(seed):
    """rand(*shape, scale): seeded normal values in bf16."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    return rand


def main():
    a, rand = arguments(__doc__), generator(0)
    layer = ExpertLayer(rand(a.experts, 2 * a.inner, a.hidden, scale=a.hidden ** -0.5),
                        rand(a.experts, a.hidden, a.inner, scale=a.inner ** -0.5), rand(a.experts, a.hidden, scale=a.hidden ** -0.5),
                        a.topk)
    x, dy = rand(a.tokens, a.hidden), rand(a.tokens, a.hidden)
    y, kept = layer.forward(x)
    layer.backward(dy, kept)
    if int(kept["plan"]["d_status"]):
        raise RuntimeError("the plan did not fit its capacity")
    print(f"forward  {a.tokens} tokens: {timed(lambda: layer.forward(x)):9.1f} us")
    print(f"backward {a.tokens} tokens: {timed(lambda: layer.backward(dy, kept)):9.1f} us")
    few = x[:4].contiguous()
    print(f"decode   {few.shape[0]} tokens:    {timed(lambda: layer.decode(few)):9.1f} us")
    adapters, rank = 6, 16
    project = AdaptedProjection(rand(a.hidden, a.hidden, scale=a.hidden ** -0.5), rand(adapters, rank, a.hidden, scale=a.hidden ** -0.5),
                                rand(adapters, a.hidden, rank, scale=rank ** -0.5), torch.ones(adapters, device="cuda"))
    ids = torch.tensor([0, 5, -1, 3], dtype=torch.int32, device="cuda")
    print(f"project  {few.shape[0]} tokens:    {timed(lambda: project(few, ids)):9.1f} us")


if __name__ == "__main__":
    main()
