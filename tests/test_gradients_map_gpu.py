"""Dispatch's gradient where it rebuilds the pick -> row map: many picks (more than 8192) of short rows that align to 16
bytes, in a workspace that has no map of them. (Smaller batches, longer rows and combine's gradient look for their
rows instead, also in a fresh workspace.)"""
import numpy as np
import pytest
import torch

from test_gradients_gpu import Routed

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import moe as M

# W, bs, K, E, h, Z, C, mask, dtype; W * bs * K above 8192 and rows below 8192 bytes
CASES = [
    (4, 600, 4, 16, 64, 1, 2, 2, "bf16"),
    (2, 700, 6, 8, 8, 0, 0, 0, "f16"),
    (8, 150, 8, 32, 520, 2, 0, 1, "f16"),
    (2, 2100, 2, 4, 4088, 0, 1, 2, "bf16"),
]
ids_of = lambda c: "-".join(map(str, c))  # noqa: E731


def backward(r, y, ws, residual=None, row_weights=None, in_place=False, launches=2):
    """dispatch_backward, and that it went the way that is meant: the map and the reduce, or the reduce alone."""
    before = M.launch_count()
    got = r.dispatch_backward(y, residual, row_weights, in_place, ws)
    assert M.launch_count() - before == launches
    return got


@pytest.mark.parametrize("case", CASES, ids=ids_of)
def test_rebuilt_map(case):
    r = Routed(*case, seed=sum(case[:5]))
    y, y64 = r.expert_rows()
    res, res64 = r.rows((r.W, r.bs, r.h))
    rw = torch.randn(r.W, r.A, device="cuda")
    fresh = M.alloc_workspace(r.cfg)
    got = backward(r, y, fresh, res, rw)
    r.check_dispatch(got, y64, res64, rw)
    # byte for byte what the dispatch's own map gives
    own = backward(r, y, r.ws, res, rw, launches=1)
    assert torch.equal(got[0], own[0]) and torch.equal(got[1], own[1])
    # once more, in place, and without a residual
    assert torch.equal(got[0], backward(r, y, fresh, res.clone(), in_place=True)[0])
    r.check_dispatch(backward(r, y, fresh), y64)


def test_rows_in_another_order():
    r = Routed(*CASES[0], seed=4)
    y, y64 = r.expert_rows()
    g, g64 = r.rows((r.W, r.bs, r.h))
    rw = torch.randn(r.W, r.A, device="cuda")
    order = np.tile(np.arange(r.A), (r.W, 1))
    for d in range(r.W):
        edges = [0, *r.ep[d]]
        for lo, hi in zip(edges[:-1], edges[1:]):
            order[d, lo:hi] = lo + r.rng.permutation(hi - lo)
    r.assist = np.take_along_axis(r.assist, order[..., None], 1)
    r.out["assist_info"] = torch.from_numpy(r.assist).cuda()  # in a buffer of its own: no map is its
    r.where = {tuple(r.assist[d, i]): (d, i) for d in range(r.W) for i in range(r.ep[d, -1])}
    r.check_dispatch(backward(r, y, r.ws, g, rw), y64, g64, rw)


def test_reports_rows_that_do_not_match():
    def status(change):
        r = Routed(4, 600, 4, 16, 64, seed=5)
        change(r)
        y = torch.zeros(r.W, r.A, r.h, dtype=torch.bfloat16, device="cuda")
        gx, ws = torch.empty(r.W, r.bs, r.h, dtype=torch.bfloat16, device="cuda"), M.alloc_workspace(r.cfg)
        before = M.launch_count()
        M.dispatch_backward(r.cfg, y, *r.route(), None, gx, ws=ws)
        assert M.launch_count() - before == 2
        return M.STATUS[M.get_device_status(ws)]

    assert status(lambda r: None) == "OK"
    assert status(lambda r: r.out["assist_info"][0, 1].fill_(-1)) == "BAD_ASSIST"
    assert status(lambda r: r.out["assist_info"][2, 7, 2].fill_(4)) == "BAD_ASSIST"
    assert status(lambda r: r.out["ep_recv_count"][1, -1:].sub_(1)) == "BAD_ASSIST"
    assert status(lambda r: r.out["ep_recv_count"][1, -1:].fill_(r.A + 1)) == "BAD_ASSIST"
    assert status(lambda r: r.ids_d[1, 2, 0].fill_(16)) == "BAD_EXPERT_ID"
    assert status(lambda r: r.ids_d[1, 2].copy_(r.ids_d[1, 2].flip(0))) == "BAD_ASSIST"


def test_captured_and_replayed_beside_other_dispatches():
    """Two batches of one workspace: the graph's gradient of the one rebuilds its map, whatever was dispatched before, and
    leaves none that the other one's calls would take for theirs."""
    a, b = Routed(*CASES[0], seed=10), Routed(*CASES[0], seed=11)
    ya, ya64 = a.expert_rows()
    yb, yb64 = b.expert_rows()
    rb = torch.randn(b.W, b.A, device="cuda")
    want_a, want_b = a.dispatch_backward(ya)[0], b.dispatch_backward(yb, None, rb)
    combined = torch.empty_like(b.x)

    def combine(out):
        M.combine(b.cfg, yb, b.out["assist_info"], b.out["ep_recv_count"], b.ids_d, b.weights_d, b.mask, b.x, out, None, ws)

    ws = b.ws
    combine(combined)
    sums, got = torch.full_like(want_a, 7.0), torch.full_like(combined, 7.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.dispatch_backward(a.cfg, ya, *a.route(), a.mask, sums, ws=ws)
    for _ in range(2):
        sums.fill_(7.0), got.fill_(7.0)
        M.dispatch(b.cfg, b.x, b.ids_d, b.mask, b.weights_d, b.out["expand_x"], None, b.out["assist_info"], b.out["ep_recv_count"],
                   b.out["expand_scales"], None, ws)
        graph.replay()
        combine(got)
        again = b.dispatch_backward(yb, None, rb)
        assert M.get_device_status(ws) == 0
        assert torch.equal(sums, want_a) and torch.equal(got, combined)
        assert torch.equal(again[0], want_b[0]) and torch.equal(again[1], want_b[1])
    a.check_dispatch((sums, None), ya64)
    b.check_dispatch(again, yb64, None, rb)


def test_the_backward_of_two_micro_batches():
    """Forward, forward, backward, backward on one workspace, eagerly, and a combine after each gradient."""
    a, b = Routed(*CASES[0], seed=20), Routed(*CASES[0], seed=21)
    ws = a.ws
    made = []
    for r in (a, b):
        y, y64 = r.expert_rows()
        out = torch.empty_like(r.x)
        M.combine(r.cfg, y, r.out["assist_info"], r.out["ep_recv_count"], r.ids_d, r.weights_d, r.mask, r.x, out, None, r.ws)
        made.append((r, y, y64, out))
    for r in (a, b):
        M.dispatch(r.cfg, r.x, r.ids_d, r.mask, r.weights_d, r.out["expand_x"], None, r.out["assist_info"], r.out["ep_recv_count"],
                   r.out["expand_scales"], None, ws)
    for n, (r, y, y64, out) in enumerate((made[1], made[0], made[1])):
        r.check_dispatch(backward(r, y, ws, launches=2 if n else 1), y64)
        again = torch.empty_like(out)
        M.combine(r.cfg, y, r.out["assist_info"], r.out["ep_recv_count"], r.ids_d, r.weights_d, r.mask, r.x, again, None, ws)
        assert M.get_device_status(ws) == 0 and torch.equal(again, out)


def test_a_step_in_one_graph_on_one_workspace():
    """Dispatch, combine and both gradients captured together: by the dispatch's own map, whatever another batch's calls
    leave in the workspace between the replays."""
    a, b = Routed(*CASES[0], seed=30), Routed(*CASES[0], seed=31)
    ya, ya64 = a.expert_rows()
    yb, _ = b.expert_rows()
    g, g64 = a.rows((a.W, a.bs, a.h))
    want, want_b = a.combine_backward(g, ya, x=True), b.dispatch_backward(yb)[0]
    gx = a.dispatch_backward(ya, g)[0]
    ws = a.ws
    rows, weights, x, sums = (torch.full_like(t, 7.0) for t in (*want.values(), gx))
    result, eager = torch.empty_like(a.x), torch.empty_like(a.x)

    def combine(out, space):
        M.combine(a.cfg, ya, a.out["assist_info"], a.out["ep_recv_count"], a.ids_d, a.weights_d, a.mask, a.x, out, None, space)

    combine(eager, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = M.launch_count()
    with torch.cuda.graph(graph):
        M.dispatch(a.cfg, a.x, a.ids_d, a.mask, a.weights_d, a.out["expand_x"], None, a.out["assist_info"], a.out["ep_recv_count"],
                   a.out["expand_scales"], None, ws)
        combine(result, ws)
        M.combine_backward(a.cfg, g, ya, *a.route(), a.weights_d, a.mask, a.x, rows, weights, x, ws)
        M.dispatch_backward(a.cfg, ya, *a.route(), a.mask, sums, g, ws=ws)
    assert M.launch_count() - before == 5  # routing and scatter, then one each
    for _ in range(2):
        for t in (rows, weights, x, sums, result):
            t.fill_(7.0)
        again = b.dispatch_backward(yb, ws=ws)[0]  # rebuilds the map for its own rows
        graph.replay()
        torch.cuda.synchronize()
        assert M.get_device_status(ws) == 0 and torch.equal(again, want_b)
        assert torch.equal(rows, want["rows"]) and torch.equal(weights, want["weights"]) and torch.equal(x, want["x"])
        assert torch.equal(sums, gx) and torch.equal(result, eager)
    a.check_combine(dict(rows=rows, weights=weights, x=x), g64, ya64)
    a.check_dispatch((sums, None), ya64, g64)
