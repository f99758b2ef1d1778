"""A decode MoE layer on int8 experts, from router logits to the layer's output:

    route -> dispatch (int8 rows, a scale each) -> gate/up product with SwiGLU
          -> int8 rows again -> down product -> combine

Every step is one call of the library (``combine_route_scan_gb300.moe``). The weights
are quantised once, when the layer is made, with a scale for each output channel.
Every token is active and every expert one of the E: the dispatch's token masks and
its zero and copy experts are not passed on.

``python -m combine_route_scan_gb300.int8_layer`` builds one on random weights
(8 ranks x 64 tokens, hidden 2048, 128 experts, top-8, intermediate 512), runs
it next to the bf16 layer call (moe_dispatch_ffn_combine) and prints the times
and how far the two outputs are apart.
"""
from __future__ import annotations

import argparse

import torch

from . import moe as M
from .routed_layer import RoutedLayer, compare_with_bf16


class Int8Layer(RoutedLayer):
    """w_gate, w_up [E, I, h] and w_down [E, h, I] (float32, float16 or bfloat16, one
    output feature a row) for W ranks of bs tokens; bias: the router's fp32 [E]
    or None; `router` goes to moe.router_config (score_func, group_num, ...)."""

    def __init__(self, W: int, bs: int, topk: int, w_gate, w_up, w_down, bias=None, dtype=torch.bfloat16, router=None,
                 logits_dtype=torch.float32):
        E, I, h = w_gate.shape
        super().__init__(M.config(W, bs, h, topk, E, dtype, quant_mode=2), dtype, bias, router, logits_dtype, w_gate.device)
        gate_up = self.interleaved(w_gate, w_up)
        self.gate_up = M.alloc_int8(gate_up)
        M.int8_quantize(gate_up, *self.gate_up)
        self.down = M.alloc_int8(w_down)
        M.int8_quantize(w_down.contiguous(), *self.down)
        self.h1 = torch.empty((W, self.y.shape[1], I), dtype=dtype, device=w_gate.device)
        self.h1_rows = M.alloc_int8(self.h1)

    def experts(self, r):
        ep = r["ep_recv_count"]
        M.expert_product_int8(self.cfg, r["expand_x"], r["dynamic_scales"], ep, *self.gate_up, self.h1, M.EPI_SWIGLU, self.ws)
        M.int8_quantize(self.h1, *self.h1_rows, ep_recv_count=ep)
        M.expert_product_int8(self.cfg, *self.h1_rows, ep, *self.down, self.y, ws=self.ws)


def main(argv=None):
    compare_with_bf16(Int8Layer, "int8", "8-bit", argparse.ArgumentParser(
        description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter), argv)


if __name__ == "__main__":
    main()
