"""What the decode layers on quantised experts (mxfp4_layer.py, int8_layer.py) share:
the router, dispatch, combine and their gradients, with the experts between them
left to the layer, and a comparison with the bf16 layer call.
"""
from __future__ import annotations

import statistics

import torch

from . import moe as M


class RoutedLayer:
    """cfg: the dispatch's configuration. A layer brings ``experts(rows)``, which takes the
    dispatched rows (a dict as of moe.alloc_dispatch_outputs) to ``self.y`` [W, A, h]."""

    def __init__(self, cfg, dtype, bias, router, logits_dtype, device):
        W, bs, h, K, E = cfg.ep_world_size, cfg.bs, cfg.h, cfg.topk, cfg.moe_expert_num
        self.cfg = cfg
        self.combine_cfg = M.config(W, bs, h, K, E, dtype)
        self.router = M.router_config(W * bs, E, K, logits_dtype, **(router or {}))
        self.bias = bias
        # what a step writes on its way, kept for the next one
        self.ws = M.alloc_workspace(self.cfg)
        _, A = M.workspace_size(self.cfg)
        self.rows = M.alloc_dispatch_outputs(self.cfg, dtype, expand_scales=False)
        self.y = torch.empty((W, A, h), dtype=dtype, device=device)
        self.ids = torch.empty((W, bs, K), dtype=torch.int32, device=device)
        self.weights = torch.empty((W, bs, K), dtype=torch.float32, device=device)

    @staticmethod
    def interleaved(w_gate, w_up):
        """The rows of gate and up in turns, as the products' SwiGLU wants them."""
        E, I, h = w_gate.shape
        return torch.stack((w_gate, w_up), 2).reshape(E, 2 * I, h)

    def __call__(self, x, logits, out=None):
        """x [W, bs, h], logits [W * bs, E] -> the layer's output [W, bs, h]. Device
        errors are read with moe.get_device_status(layer.ws)."""
        out = torch.empty_like(x) if out is None else out
        r = self.rows
        M.route(self.router, logits, self.bias, self.ids, self.weights)
        M.dispatch(self.cfg, x, self.ids, None, None, r["expand_x"], r["dynamic_scales"], r["assist_info"],
                   r["ep_recv_count"], None, None, self.ws)
        self.experts(r)
        M.combine(self.combine_cfg, self.y, r["assist_info"], r["ep_recv_count"], self.ids, self.weights, None, x, out,
                  None, self.ws)
        return out

    def weights_gradient(self, grad_out, out=None):
        """The gradient of the last step's routing weights, from that of its output: how much each chosen
        expert's answer would have helped."""
        out = torch.empty_like(self.weights) if out is None else out
        r = self.rows
        M.combine_backward(self.combine_cfg, grad_out, self.y, r["assist_info"], r["ep_recv_count"], self.ids, self.weights,
                           None, None, None, out, ws=self.ws)
        return out

    def logits_gradient(self, logits, grad_weights, out=None):
        """The gradient of the last step's routing weights with respect to its logits, from the loss's gradient by those
        weights (weights_gradient)."""
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


def compare_with_bf16(layer_type, name, rounding, ap, argv=None):
    """A layer on random weights next to the bf16 layer call: times, and how far the two outputs are apart."""
    for flag, value in (("ranks", 8), ("bs", 64), ("h", 2048), ("experts", 128), ("topk", 8), ("intermediate", 512)):
        ap.add_argument("--" + flag, type=int, default=value)
    ap.add_argument("--reps", type=int, default=50)
    a = ap.parse_args(argv)
    W, bs, h, E, K, I = a.ranks, a.bs, a.h, a.experts, a.topk, a.intermediate
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *shape, std=1.0: (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    w_gate, w_up, w_down = draw(E, I, h, std=0.02), draw(E, I, h, std=0.02), draw(E, h, I, std=0.02)
    x, logits = draw(W, bs, h), torch.randn(W * bs, E, generator=g, device="cuda")
    layer = layer_type(W, bs, K, w_gate, w_up, w_down)
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
    print(f"{name + ' layer, routing included:':33s}{_time(lambda: layer(x, logits, out), a.reps):8.1f} us")
    print(f"{'bf16 layer call:':33s}{_time(bf16, a.reps):8.1f} us")
    print(f"relative difference of the outputs (the {rounding} rounding of rows and weights): {off:.3f}")
