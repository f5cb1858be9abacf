#!/usr/bin/env python3
"""A mixture-of-experts layer with 8-bit integer weights, at decode and at prefill.

One set of weights (int8 codes, one scale per output channel) serves both:

  decode   gate -> the whole layer in one kernel (at most 64 tokens; activations stay bf16)
  prefill  gate -> dispatch into the experts' planes -> rows to int8 -> product -> SiLU * up
           -> rows to int8 -> product into the combine payload -> gated combine

    python examples/int8_moe.py            # needs a GB300 and the built library
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from combine_topk_ids_rank_gb300 import moe_a2a as moe  # noqa: E402


class Int8MoE:
    """Router and experts of one layer; `ranks` x `max_tokens` tokens at most at prefill."""

    def __init__(self, ranks, max_tokens, hidden, inter, experts, top_k, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.top_k, self.hidden, self.experts, self.ranks = top_k, hidden, experts, ranks

        def weights(out, inner):
            w = torch.randn((experts, out, inner), generator=g, device=device) / inner ** 0.5
            return moe.quantize_rows_int8(w)            # codes and a scale per output channel

        self.router = torch.randn((hidden, experts), generator=g, device=device) / hidden ** 0.5
        self.w13, self.s13 = weights(2 * inter, hidden)
        self.w2, self.s2 = weights(hidden, inter)
        self.few = moe.MoeLayerSmall(experts, hidden, inter, top_k, moe.MOE_LAYER_MAX_TOKENS,
                                     moe.MOE_FORMAT_INT8, device)
        self.a2a = moe.MoeA2A(ranks, max_tokens, hidden, experts, top_k, device,
                              layout=moe.MOE_LAYOUT_EXPERT)
        rows = ranks * max_tokens
        self.up = moe.MoeGemmInt8(experts, rows, 2 * inter, hidden, device)
        self.down = moe.MoeGemmInt8(experts, rows, hidden, inter, device)

    def gate(self, x):
        return moe.topk_gate(x.float() @ self.router, self.top_k, moe.MOE_SCORE_SOFTMAX)

    def decode(self, x):
        """x bf16 [tokens, hidden], at most 64 tokens."""
        ids, w = self.gate(x)
        return self.few.forward(x, ids, w, self.w13, self.w2, self.s13, self.s2)

    def prefill(self, x):
        """x bf16 [ranks, tokens, hidden]."""
        ids, w = self.gate(x)
        view = self.a2a.dispatch(ids, w, x)
        counts = view.recv_counts                       # rows of each expert, on the device
        xq, sx = moe.quantize_rows_int8(view.recv_x, counts)
        gate, up = self.up.gemm(xq, sx, self.w13, self.s13, counts).chunk(2, -1)
        act = torch.nn.functional.silu(gate) * up
        aq, sa = moe.quantize_rows_int8(act, counts)
        self.down.gemm(aq, sa, self.w2, self.s2, counts, out=self.a2a.combine_payload())
        return self.a2a.combine(None, True)


def reference(layer, x):
    """The layer on its dequantised weights in 64 bits; x bf16 [tokens, hidden]."""
    ids, w = layer.gate(x)
    X, out = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(layer.experts):
        t, k = (ids == e).nonzero(as_tuple=True)
        if len(t):
            h = X[t] @ (layer.w13[e].double() * layer.s13[e].double()[:, None]).T
            gate, up = h.chunk(2, -1)
            a = gate * torch.sigmoid(gate) * up
            y = a @ (layer.w2[e].double() * layer.s2[e].double()[:, None]).T
            out.index_add_(0, t, y * w[t, k].double()[:, None])
    return out


def main(ranks=4, tokens=96, hidden=1024, inter=512, experts=16, top_k=4):
    layer = Int8MoE(ranks, tokens, hidden, inter, experts, top_k)
    x = torch.randn((ranks, tokens, hidden), device="cuda").to(torch.bfloat16)
    y = layer.prefill(x).reshape(ranks * tokens, hidden)
    flat = x.reshape(ranks * tokens, hidden)
    ref = reference(layer, flat)
    few = flat[:: ranks * tokens // 48][:48].contiguous()
    z, zref = layer.decode(few), reference(layer, few)
    torch.cuda.synchronize()
    for h in (layer.a2a, layer.few, layer.up, layer.down):
        assert h.get_error() == (0, 0)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    errors = {"prefill": off(y, ref), "decode": off(z, zref)}
    print("relative error against 64 bits: prefill (8-bit activations) %.2e, decode (bf16) %.2e"
          % (errors["prefill"], errors["decode"]))
    return errors


if __name__ == "__main__":
    main()
