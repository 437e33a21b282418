"""The expert layer of ``moe_layer.py`` with its 8-bit operators.

    python examples/moe_layer_8bit.py [--tokens 4096] [--hidden 2048] [--inner 1024] [--experts 32] [--topk 4]

* ``KeptLayer``: the training step with the router's balance loss and with the
  gated block's checkpoint in 8 bits.  The hidden rows are not kept at all: the
  backward pass makes them again from the checkpoint;
* ``Int8Layer``: serving with the experts' weights in 8-bit integers, a scale
  for each channel, and the activations cast with a scale for each token: a
  batch in packed groups, a few tokens of decoding requests, and a shared
  expert beside the chosen ones.

Run as a program it does one step of each and prints their times.
"""
from __future__ import annotations

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)

import moe_layer  # noqa: E402
from moe_layer import B, ExpertLayer, moe, timed  # noqa: E402
from nvfp4_block_scaled_group_amd import i8  # noqa: E402


class KeptLayer(ExpertLayer):
    """ExpertLayer with a balance loss of weight ``coef``, sequence by sequence, and an 8-bit checkpoint."""

    def __init__(self, gate_up, down, router, topk, coef=0.01):
        super().__init__(gate_up, down, router, topk)
        self.coef = coef

    def forward(self, x, seq_ends=None):
        """x [T, h] bf16, seq_ends [S] i32 -> y [T, h] bf16, the balance loss [1] f32, and what backward needs."""
        T, S = x.shape[0], 1 if seq_ends is None else seq_ends.numel()
        logits, ids, weights = self.route(x)
        balance = moe.alloc_balance(T, self.E, S, device=self.dev)
        moe.moe_balance(logits, ids, **balance, seq_ends=seq_ends, coef=self.coef)
        plan = moe.alloc_plan(T, self.topk, self.E, device=self.dev)
        moe.moe_plan(ids, **plan)
        cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
        packed = self._bf16(cap, self.h)
        moe.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        x_rows, x_cols = self._quantize(packed, plan)
        hidden, checkpoint = self._bf16(cap, self.f), moe.alloc_keep8(cap, self.f, device=self.dev)
        moe.moe_glu_keep8_graphsafe(*x_rows, *self.gu_lines, offs, hidden, **checkpoint, d_status=status)
        h_rows, _ = self._quantize(hidden, plan)
        out = torch.empty((cap, self.h), device=self.dev)
        B.nvfp4_group_gemm_graphsafe(*h_rows, *self.down_lines, offs, out, status)
        y = self._bf16(T, self.h)
        moe.moe_combine(out, plan["rows"], y, weights=weights)
        return y, balance["loss"], dict(logits=logits, ids=ids, weights=weights, plan=plan, x_cols=x_cols, out=out,
                                        checkpoint=checkpoint, balance=balance, seq_ends=seq_ends)

    def backward(self, dy, kept, dloss=None):
        """dy [T, h] bf16, dloss [1] f32 (None: 1) -> gradients of x (through the experts), the logits, gate_up and down."""
        T, plan, bal = dy.shape[0], kept["plan"], kept["balance"]
        cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
        d_out, dw = self._bf16(cap, self.h), torch.empty((T, self.topk), device=self.dev)
        moe.moe_dispatch(dy, plan["rows"], plan["src"], offs, d_out, weights=kept["weights"], y=kept["out"], dweights=dw)
        # the logits have two gradients: through the weights, and through the balance loss
        dlogits = torch.empty_like(kept["logits"])
        moe.moe_route_bwd(kept["logits"], kept["ids"], dw, dlogits)
        moe.moe_balance_bwd(kept["logits"], bal["counts"], bal["seq_tokens"], dlogits, topk=self.topk,
                            seq_ends=kept["seq_ends"], coef=self.coef, dloss=dloss, add=dlogits)
        do_rows, do_cols = self._quantize(d_out, plan)
        dgu, hidden = self._bf16(cap, self.f2), self._bf16(cap, self.f)
        moe.moe_glu_bwd_keep8_graphsafe(*do_rows, *self.down_turned, offs, **kept["checkpoint"], dgu=dgu, d_status=status,
                                        h=hidden)
        _, h_cols = self._quantize(hidden, plan)
        d_down = torch.empty((self.E, self.h, self.f), device=self.dev)
        B.nvfp4_group_gemm_wgrad_graphsafe(*do_cols, *h_cols, cap, self.E, offs, self.h, self.f, d_down, status)
        dgu_rows, dgu_cols = self._quantize(dgu, plan)
        d_packed = torch.empty((cap, self.h), device=self.dev)
        B.nvfp4_group_gemm_graphsafe(*dgu_rows, *self.gu_turned, offs, d_packed, status)
        d_gu = torch.empty((self.E, self.f2, self.h), device=self.dev)
        B.nvfp4_group_gemm_wgrad_graphsafe(*dgu_cols, *kept["x_cols"], cap, self.E, offs, self.f2, self.h, d_gu, status)
        dx = self._bf16(T, self.h)
        moe.moe_combine(d_packed, plan["rows"], dx)
        return dx, dlogits, d_gu, d_down


def cast_channels(w):
    """bf16 weights [..., k] -> int8 codes [..., k] and a scale for each channel [...]."""
    made = i8.alloc_cast(w.numel() // w.shape[-1], w.shape[-1], device=w.device)
    i8.i8_group_cast(w.view(-1, w.shape[-1]), **made)
    return made["q"].view(w.shape), made["scale"].view(w.shape[:-1])


class Int8Layer:
    """Serving: gate_up [E, 2f, h], down [E, h, f], router [E, h], shared [h, h] (a projection that every token passes)."""

    def __init__(self, gate_up, down, router, shared, topk):
        self.E, f2, self.h = gate_up.shape
        self.f, self.topk, self.router, self.dev = f2 // 2, topk, router.float(), gate_up.device
        self.gate_up, self.down, self.shared = cast_channels(gate_up), cast_channels(down), cast_channels(shared)

    def _bf16(self, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=self.dev)

    route = ExpertLayer.route

    def _cast(self, x):
        made = i8.alloc_cast(*x.shape, device=self.dev)
        i8.i8_group_cast(x, **made)
        return made["q"], made["scale"]

    def _cast_packed(self, x, plan):
        made = i8.alloc_cast(*x.shape, device=self.dev)
        i8.i8_group_cast_graphsafe(x, plan["d_offs"], **made, d_status=plan["d_status"])
        return made["q"], made["scale"]

    def project(self, x):
        """The shared projection of x [T, h], any number of rows."""
        y = self._bf16(x.shape[0], self.h)
        ws = torch.empty(i8.i8_linear_workspace(x.shape[0], self.h, self.h), dtype=torch.uint8, device=self.dev)
        i8.i8_linear(*self._cast(x), *self.shared, y, ws)
        return y

    def batch(self, x):
        """x [T, h] bf16 of prompts -> y [T, h] bf16."""
        T = x.shape[0]
        _, ids, weights = self.route(x)
        plan = moe.alloc_plan(T, self.topk, self.E, device=self.dev)
        moe.moe_plan(ids, **plan)
        cap, offs, status = plan["src"].numel(), plan["d_offs"], plan["d_status"]
        packed, hidden = self._bf16(cap, self.h), self._bf16(cap, self.f)
        moe.moe_dispatch(x, plan["rows"], plan["src"], offs, packed)
        i8.i8_group_glu_graphsafe(*self._cast_packed(packed, plan), *self.gate_up, offs, hidden, status)
        out, y = self._bf16(cap, self.h), self._bf16(T, self.h)
        i8.i8_group_gemm_graphsafe(*self._cast_packed(hidden, plan), *self.down, offs, out, status)
        moe.moe_combine(out, plan["rows"], y, weights=weights)
        return y + self.project(x)

    def decode(self, x):
        """x [T, h] bf16 of a few requests -> y [T, h] bf16."""
        T = x.shape[0]
        _, ids, weights = self.route(x)
        hidden = self._bf16(T * self.topk, self.f)
        i8.i8_token_glu(x, ids, *self.gate_up, hidden)
        out = torch.empty((T * self.topk, self.h), device=self.dev)
        i8.i8_token_linear(hidden, ids, *self.down, out)
        rows = torch.arange(T * self.topk, dtype=torch.int32, device=self.dev).view(T, self.topk)
        y = self._bf16(T, self.h)
        moe.moe_combine(out, rows, y, weights=weights)
        return y + self.project(x)


def main():
    a = moe_layer.arguments(__doc__)
    rand = moe_layer.generator(0)
    gate_up = rand(a.experts, 2 * a.inner, a.hidden, scale=a.hidden ** -0.5)
    down, router = rand(a.experts, a.hidden, a.inner, scale=a.inner ** -0.5), rand(a.experts, a.hidden, scale=a.hidden ** -0.5)
    x, dy = rand(a.tokens, a.hidden), rand(a.tokens, a.hidden)
    ends = torch.tensor([a.tokens // 3, a.tokens // 2, a.tokens], dtype=torch.int32, device="cuda")
    layer = KeptLayer(gate_up, down, router, a.topk)
    y, loss, kept = layer.forward(x, ends)
    layer.backward(dy, kept)
    if int(kept["plan"]["d_status"]):
        raise RuntimeError("the plan did not fit its capacity")
    print(f"forward  {a.tokens} tokens: {timed(lambda: layer.forward(x, ends)):9.1f} us, balance loss {float(loss):.4f}")
    print(f"backward {a.tokens} tokens: {timed(lambda: layer.backward(dy, kept)):9.1f} us")
    served = Int8Layer(gate_up, down, router, rand(a.hidden, a.hidden, scale=a.hidden ** -0.5), a.topk)
    few = x[:4].contiguous()
    print(f"batch    {a.tokens} tokens: {timed(lambda: served.batch(x)):9.1f} us")
    print(f"decode   {few.shape[0]} tokens:    {timed(lambda: served.decode(few)):9.1f} us")


if __name__ == "__main__":
    main()
