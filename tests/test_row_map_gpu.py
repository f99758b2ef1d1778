"""The pick -> row map that a workspace keeps from its last dispatch: a combine of other
buffers replaces it, eagerly or by the replay of a graph, and is not taken for that dispatch's."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import workloads as WL

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()


def batches():
    """Two batches of one shape, their dispatches' outputs (each by a workspace of its own) and combined rows."""
    made = []
    for seed in (1, 2):
        wl = WL.Workload(f"map{seed}", 2, 24, 64, 3, 8, WL.X_INT32, seed=seed)
        dev = H.device_inputs(wl, WL.make_inputs(wl))
        out, _, _ = H.gpu_dispatch(wl, dev)
        want, _, _ = H.gpu_combine(wl, dev, out["expand_x"], out["assist_info"], out["ep_recv_count"])
        made.append((wl, dev, out, want))
    return made


def combine(batch, ws, x_out):
    wl, dev, out, _ = batch
    M.combine(H.make_cfg(wl), out["expand_x"], out["assist_info"], out["ep_recv_count"], dev["expert_ids"], dev["expert_scales"],
              None, dev["x"], x_out, None, ws)


def test_a_combine_of_other_rows_leaves_the_dispatch_no_map():
    a, b = batches()
    ws = M.alloc_workspace(H.make_cfg(a[0]))
    H.gpu_dispatch(b[0], b[1], ws=ws, out=b[2])  # its map is the workspace's
    for batch in (b, a, b, b, a, a, b):
        got = torch.zeros_like(batch[3])
        combine(batch, ws, got)
        assert M.get_device_status(ws) == 0 and torch.equal(got, batch[3])


def test_a_replayed_combine_of_other_rows():
    a, b = batches()
    ws = M.alloc_workspace(H.make_cfg(a[0]))
    got_a, got_b = torch.zeros_like(a[3]), torch.zeros_like(b[3])
    combine(a, ws, got_a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        combine(a, ws, got_a)
    for _ in range(2):
        H.gpu_dispatch(b[0], b[1], ws=ws, out=b[2])
        graph.replay()
        combine(b, ws, got_b)
        assert M.get_device_status(ws) == 0
        assert torch.equal(got_a, a[3]) and torch.equal(got_b, b[3])


def test_another_combine_captured_between_a_dispatch_and_its_own():
    a, b = batches()
    ws = M.alloc_workspace(H.make_cfg(a[0]))
    got_a, got_b = torch.zeros_like(a[3]), torch.zeros_like(b[3])
    cfg = H.make_cfg(b[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        M.dispatch(cfg, b[1]["x"], b[1]["expert_ids"], None, b[1]["expert_scales"], b[2]["expand_x"], None, b[2]["assist_info"],
                   b[2]["ep_recv_count"], b[2]["expand_scales"], None, ws)
        combine(a, ws, got_a)
        combine(b, ws, got_b)
    for _ in range(2):
        graph.replay()
        assert M.get_device_status(ws) == 0
        assert torch.equal(got_a, a[3]) and torch.equal(got_b, b[3])
        got_a.zero_(), got_b.zero_()
