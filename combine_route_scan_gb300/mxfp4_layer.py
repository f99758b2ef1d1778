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
import statistics

import torch

from . import moe as M


class Mxfp4Layer:
    """w_gate, w_up [E, I, h] and w_down [E, h, I] (float32, float16 or bfloat16, one
    output feature a row) for W ranks of bs tokens; bias: the router's fp32 [E]
    or None; `router` goes to moe.router_config (score_func, group_num, ...)."""

    def __init__(self, W: int, bs: int, topk: int, w_gate, w_up, w_down, bias=None, dtype=torch.bfloat16, router=None,
                 logits_dtype=torch.float32):
        E, I, h = w_gate.shape
        self.cfg = M.config(W, bs, h, topk, E, dtype, quant_mode=4, expand_dtype="fp4_e2m1")
        self.combine_cfg = M.config(W, bs, h, topk, E, dtype)
        self.router = M.router_config(W * bs, E, topk, logits_dtype, **(router or {}))
        self.bias = bias
        # the rows of gate and up take turns, as the product's SwiGLU wants them
        gate_up = torch.stack((w_gate, w_up), 2).reshape(E, 2 * I, h)
        self.gate_up = M.alloc_mx(gate_up, M.SF_TILED)
        M.mx_quantize(gate_up, *self.gate_up, layout=M.SF_TILED)
        self.down = M.alloc_mx(w_down, M.SF_TILED)
        M.mx_quantize(w_down.contiguous(), *self.down, layout=M.SF_TILED)
        # what a step writes on its way, kept for the next one
        self.ws = M.alloc_workspace(self.cfg)
        _, A = M.workspace_size(self.cfg)
        dev = w_gate.device
        self.rows = M.alloc_dispatch_outputs(self.cfg, dtype, expand_scales=False)
        self.h1 = torch.empty((W, A, I // 2), dtype=torch.uint8, device=dev)
        self.h1_scales = torch.empty((W, A, -(-I // 32)), dtype=torch.uint8, device=dev)
        self.y = torch.empty((W, A, h), dtype=dtype, device=dev)
        self.ids = torch.empty((W, bs, topk), dtype=torch.int32, device=dev)
        self.weights = torch.empty((W, bs, topk), dtype=torch.float32, device=dev)

    def __call__(self, x, logits, out=None):
        """x [W, bs, h], logits [W * bs, E] -> the layer's output [W, bs, h]. Device
        errors are read with moe.get_device_status(layer.ws)."""
        out = torch.empty_like(x) if out is None else out
        r = self.rows
        M.route(self.router, logits, self.bias, self.ids, self.weights)
        M.dispatch(self.cfg, x, self.ids, None, None, r["expand_x"], r["dynamic_scales"], r["assist_info"],
                   r["ep_recv_count"], None, None, self.ws)
        M.expert_product(self.cfg, r["expand_x"], r["dynamic_scales"], r["ep_recv_count"], *self.gate_up, self.h1,
                         self.h1_scales, M.EPI_SWIGLU, self.ws)
        M.expert_product(self.cfg, self.h1, self.h1_scales, r["ep_recv_count"], *self.down, self.y, ws=self.ws)
        M.combine(self.combine_cfg, self.y, r["assist_info"], r["ep_recv_count"], self.ids, self.weights, None, x, out,
                  None, self.ws)
        return out

    def logits_gradient(self, logits, grad_weights, out=None):
        """The gradient of the last step's routing weights with respect to its logits. grad_weights, the
        loss's gradient by those weights, is the caller's: the library has no backward of the combine."""
        out = torch.empty_like(logits) if out is None else out
        M.route_backward(self.router, logits, self.ids, grad_weights, out)
        return out


def _time(call, reps: int) -> float:
    """Median microseconds of a call replayed from a CUDA graph."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    spans = []
    for _ in range(reps + 3):
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        stop.record()
        torch.cuda.synchronize()
        spans.append(start.elapsed_time(stop) * 1e3)
    return statistics.median(spans[3:])


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 8), ("bs", 64), ("h", 2048), ("experts", 128), ("topk", 8), ("intermediate", 512)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--reps", type=int, default=50)
    a = ap.parse_args(argv)
    W, bs, h, E, K, I = a.ranks, a.bs, a.h, a.experts, a.topk, a.intermediate
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *shape, std=1.0: (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    w_gate, w_up, w_down = draw(E, I, h, std=0.02), draw(E, I, h, std=0.02), draw(E, h, I, std=0.02)
    x, logits = draw(W, bs, h), torch.randn(W * bs, E, generator=g, device="cuda")
    layer = Mxfp4Layer(W, bs, K, w_gate, w_up, w_down)
    out = layer(x, logits)
    assert M.get_device_status(layer.ws) == 0
    cfg = M.config(W, bs, h, K, E, torch.bfloat16, ffn_intermediate=I)
    ws = M.alloc_workspace(cfg)
    want = torch.empty_like(x)
    bf16 = lambda: M.dispatch_ffn_combine(cfg, x, layer.ids, None, layer.weights, w_gate, w_up, w_down, want, ws)  # noqa: E731
    bf16()
    assert M.get_device_status(ws) == 0
    off = float((out.float() - want.float()).norm() / want.float().norm())
    print(f"{W} ranks x {bs} tokens, hidden {h}, {E} experts, top-{K}, intermediate {I}")
    print(f"MX FP4 layer, routing included: {_time(lambda: layer(x, logits, out), a.reps):8.1f} us")
    print(f"bf16 layer call:                {_time(bf16, a.reps):8.1f} us")
    print(f"relative difference of the outputs (the 4-bit rounding of rows and weights): {off:.3f}")


if __name__ == "__main__":
    main()
