"""More workspaces than the library remembers the pick -> row maps of: a graph's dispatch may still replace the map of
one that it has forgotten."""
import pytest
import torch

import gpu_harness as H
from test_row_map_gpu import batches, combine

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import moe as M


def dispatch(batch, ws):
    wl, dev, out, _ = batch
    M.dispatch(H.make_cfg(wl), dev["x"], dev["expert_ids"], None, dev["expert_scales"], out["expand_x"], None, out["assist_info"],
               out["ep_recv_count"], out["expand_scales"], None, ws)


def test_a_dispatch_replayed_behind_many_other_workspaces():
    a, b = batches()
    cfg = H.make_cfg(a[0])
    ws = M.alloc_workspace(cfg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dispatch(a, ws)
    others = [M.alloc_workspace(cfg) for _ in range(300)]
    got_a, got_b = torch.zeros_like(a[3]), torch.zeros_like(b[3])
    for _ in range(2):
        dispatch(b, ws)
        graph.replay()  # the map is now the other batch's
        combine(b, ws, got_b)
        combine(a, ws, got_a)
        assert M.get_device_status(ws) == 0
        assert torch.equal(got_a, a[3]) and torch.equal(got_b, b[3])
        got_a.zero_(), got_b.zero_()
    # a workspace that was initialised since is no graph's: its own dispatch's map is taken as it is
    dispatch(b, others[-1])
    before = M.launch_count()
    combine(b, others[-1], got_b)
    assert M.launch_count() - before == 1 and torch.equal(got_b, b[3])
