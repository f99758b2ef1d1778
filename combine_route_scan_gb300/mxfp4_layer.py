"""A decode MoE layer on MX FP4 experts, from router logits to the layer's output:

    route -> dispatch (FP4 rows) -> gate/up product with SwiGLU (FP4 rows out)
          -> down product -> combine

Every step is one call of the library (``combine_route_scan_gb300.moe``); the
rows stay in 4 bits from the dispatch to the down projection. The weights are
quantised once, when the layer is made. Every token is active and every expert one
of the E: the dispatch's token masks and its zero and copy experts are not passed on.

``python -m combine_route_scan_gb300.mxfp4_layer`` builds one on random weights
(8 ranks x 64 tokens, hidden 2048, 128 experts, top-8, intermediate 512), runs
it next to the bf16 layer call (moe_dispatch_ffn_combine) and prints the times
and how far the two outputs are apart.
"""
from __future__ import annotations

import argparse

import torch

from . import moe as M
from .routed_layer import RoutedLayer, compare_with_bf16


class Mxfp4Layer(RoutedLayer):
    """w_gate, w_up [E, I, h] and w_down [E, h, I] (float32, float16 or bfloat16, one
    output feature a row) for W ranks of bs tokens; bias: the router's fp32 [E]
    or None; `router` goes to moe.router_config (score_func, group_num, ...)."""

    def __init__(self, W: int, bs: int, topk: int, w_gate, w_up, w_down, bias=None, dtype=torch.bfloat16, router=None,
                 logits_dtype=torch.float32):
        E, I, h = w_gate.shape
        super().__init__(M.config(W, bs, h, topk, E, dtype, quant_mode=4, expand_dtype="fp4_e2m1"), dtype, bias, router,
                         logits_dtype, w_gate.device)
        gate_up = self.interleaved(w_gate, w_up)
        self.gate_up = M.alloc_mx(gate_up, M.SF_TILED)
        M.mx_quantize(gate_up, *self.gate_up, layout=M.SF_TILED)
        self.down = M.alloc_mx(w_down, M.SF_TILED)
        M.mx_quantize(w_down.contiguous(), *self.down, layout=M.SF_TILED)
        A = self.y.shape[1]
        self.h1 = torch.empty((W, A, I // 2), dtype=torch.uint8, device=w_gate.device)
        self.h1_scales = torch.empty((W, A, -(-I // 32)), dtype=torch.uint8, device=w_gate.device)

    def experts(self, r):
        M.expert_product(self.cfg, r["expand_x"], r["dynamic_scales"], r["ep_recv_count"], *self.gate_up, self.h1,
                         self.h1_scales, M.EPI_SWIGLU, self.ws)
        M.expert_product(self.cfg, self.h1, self.h1_scales, r["ep_recv_count"], *self.down, self.y, ws=self.ws)


def main(argv=None):
    compare_with_bf16(Mxfp4Layer, "MX FP4", "4-bit", argparse.ArgumentParser(
        description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter), argv)


if __name__ == "__main__":
    main()
