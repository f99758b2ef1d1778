"""The gradients of combine and dispatch (include/moe_experts.h) against the formulas in
64 bits and against differences, and a training step through the library's calls
against the chain rule."""
import numpy as np
import pytest
import torch

import experts_plain as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()

EPS = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 1e-40}  # half a subnormal step
CLASS_NONE, CLASS_COPY = -1, -2


class Routed:
    """A routed batch: ids with special experts and a mask, and what dispatch leaves of it."""

    def __init__(self, W, bs, K, E, h, Z=0, C=0, mask=0, dtype="bf16", seed=0):
        rng = np.random.default_rng(seed)
        self.W, self.bs, self.K, self.E, self.h, self.Z, self.C = W, bs, K, E, h, Z, C
        self.dtype = dtype
        self.cfg = M.config(W, bs, h, K, E, DT[dtype], zero_expert_num=Z, copy_expert_num=C, mask_kind=mask)
        ids = np.stack([rng.permutation(E)[:K] for _ in range(W * bs)]).reshape(W, bs, K).astype(np.int32)
        if Z + C:
            ids = np.where(rng.random(ids.shape) < 0.3, rng.integers(E, E + Z + C, ids.shape), ids).astype(np.int32)
        active = np.ones((W, bs, K), dtype=bool)
        m = None
        if mask == 1:
            m = np.arange(bs) < rng.integers(0, bs + 1, (W, 1))
            active &= m[..., None]
        elif mask == 2:
            m = rng.random((W, bs, K)) < 0.7
            m[0, 0] = False
            active &= m
        self.ids, self.cls = ids, np.where(active & (ids < E), ids, np.where(active & (ids >= E + Z), CLASS_COPY, CLASS_NONE))
        self.mask = None if m is None else torch.from_numpy(m.astype(np.uint8)).cuda()
        self.ids_d = torch.from_numpy(ids).cuda()
        self.weights = (rng.random((W, bs, K)) + 0.1).astype(np.float32)
        self.weights_d = torch.from_numpy(self.weights).cuda()
        self.rng = rng
        self.ws = M.alloc_workspace(self.cfg)
        self.out = M.alloc_dispatch_outputs(self.cfg, DT[dtype])
        self.x, self.x64 = self.rows((W, bs, h))
        M.dispatch(self.cfg, self.x, self.ids_d, self.mask, self.weights_d, self.out["expand_x"], None, self.out["assist_info"],
                   self.out["ep_recv_count"], self.out["expand_scales"], None, self.ws)
        assert M.get_device_status(self.ws) == 0
        self.assist, self.ep = self.out["assist_info"].cpu().numpy(), self.out["ep_recv_count"].cpu().numpy()
        self.A = self.assist.shape[1]
        self.where = {}  # pick -> (rank, row)
        for d in range(W):
            for r in range(self.ep[d, -1]):
                self.where[tuple(self.assist[d, r])] = (d, r)
        assert len(self.where) == (self.cls >= 0).sum()

    def rows(self, shape, fill=None):
        """Random elements of the batch's type, and what they are in 64 bits."""
        t = torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(DT[self.dtype])
        return t.cuda(), t.double().numpy()

    def expert_rows(self):
        """Random rows at the received places, NaN elsewhere."""
        t, a = self.rows((self.W, self.A, self.h))
        for d in range(self.W):
            t[d, self.ep[d, -1]:] = float("nan")
        return t, a

    def route(self):
        return self.out["assist_info"], self.out["ep_recv_count"], self.ids_d

    def combine_backward(self, grad_out, y, rows=True, weights=True, x=None, ws=None, stream=None, status=0, x_in=True):
        W, bs, K, h = self.W, self.bs, self.K, self.h
        got = dict(rows=torch.full((W, self.A, h), 7.0, dtype=DT[self.dtype], device="cuda") if rows else None,
                   weights=torch.full((W, bs, K), float("nan"), device="cuda") if weights else None,
                   x=torch.full((W, bs, h), float("nan"), dtype=DT[self.dtype], device="cuda") if x else None)
        ws = self.ws if ws is None else ws
        torch.cuda.synchronize()
        M.combine_backward(self.cfg, grad_out, y, *self.route(), self.weights_d, self.mask, self.x if x_in else None, got["rows"],
                           got["weights"], got["x"], ws, stream)
        torch.cuda.synchronize()
        assert M.get_device_status(ws) == status
        return got

    def check_combine(self, got, g64, y64):
        W, bs, K, h = self.W, self.bs, self.K, self.h
        half, tiny = HALF_ULP[self.dtype], TINY[self.dtype]
        w64 = self.weights.astype(np.float64)
        # a thread's share of a row, element after element, then lanes and warps
        terms = 8 * -(-h // 2048) + -(-h // 256) + 16
        seen = np.zeros((W, self.A), dtype=bool)
        rows = None if got["rows"] is None else got["rows"].double().cpu().numpy()
        weights = None if got["weights"] is None else got["weights"].double().cpu().numpy()
        gx = None if got["x"] is None else got["x"].double().cpu().numpy()
        for s in range(W):
            for t in range(bs):
                g, copied = g64[s, t], 0.0
                for k in range(K):
                    c = self.cls[s, t, k]
                    if c >= 0:
                        d, r = self.where[s, t, k]
                        seen[d, r] = True
                        want = w64[s, t, k] * g
                        if rows is not None:
                            assert (np.abs(rows[d, r] - want) <= (half + 2 * EPS) * np.abs(want) + tiny).all(), (s, t, k)
                        v = y64[d, r]
                    elif c == CLASS_COPY:
                        v = self.x64[s, t]
                        copied += w64[s, t, k]
                    else:
                        v = np.zeros(h)
                    if weights is not None:
                        off = abs(weights[s, t, k] - (g * v).sum())
                        assert off <= terms * EPS * np.abs(g * v).sum() + 1e-40, (s, t, k, off)
                if gx is not None:
                    want = copied * g
                    assert (np.abs(gx[s, t] - want) <= (half + (K + 2) * EPS) * np.abs(want) + tiny).all(), (s, t)
        if rows is not None:
            assert (rows[~seen] == 7.0).all()

    def dispatch_backward(self, grad_rows, residual=None, row_weights=None, in_place=False, ws=None, status=0):
        W, bs, K, h = self.W, self.bs, self.K, self.h
        gx = residual if in_place else torch.full((W, bs, h), float("nan"), dtype=DT[self.dtype], device="cuda")
        gw = torch.full((W, bs, K), float("nan"), device="cuda") if row_weights is not None else None
        ws = self.ws if ws is None else ws
        M.dispatch_backward(self.cfg, grad_rows, *self.route(), self.mask, gx, residual, row_weights, gw, ws)
        torch.cuda.synchronize()
        assert M.get_device_status(ws) == status
        return gx, gw

    def check_dispatch(self, got, y64, res64=None, row_weights=None):
        gx, gw = got[0].double().cpu().numpy(), None if got[1] is None else got[1].cpu().numpy()
        half, tiny = HALF_ULP[self.dtype], TINY[self.dtype]
        rw = None if row_weights is None else row_weights.cpu().numpy()
        for s in range(self.W):
            for t in range(self.bs):
                want = np.zeros(self.h) if res64 is None else res64[s, t].copy()
                size = np.abs(want)
                for k in range(self.K):
                    at = self.where.get((s, t, k))
                    if at is not None:
                        want, size = want + y64[at], size + np.abs(y64[at])
                    if gw is not None:
                        assert gw[s, t, k] == (rw[at] if at is not None else 0.0)
                assert (np.abs(gx[s, t] - want) <= half * np.abs(want) + (self.K + 1) * (1 + half) * EPS * size + tiny).all(), (s, t)


CASES = [
    # W, bs, K, E, h, Z, C, mask, dtype
    (2, 1, 1, 2, 1, 0, 0, 0, "bf16"),
    (2, 8, 2, 4, 256, 0, 0, 0, "f16"),
    (2, 5, 3, 6, 7, 1, 1, 2, "f16"),
    (4, 6, 4, 8, 40, 0, 2, 1, "bf16"),
    (2, 9, 8, 16, 2048, 2, 2, 2, "bf16"),
    (3, 7, 5, 9, 130, 2, 0, 0, "bf16"),
    (2, 3, 12, 32, 1032, 0, 3, 2, "f16"),
    (2, 4, 32, 64, 72, 1, 1, 2, "bf16"),
    (8, 11, 8, 128, 512, 0, 0, 1, "f16"),
    (2, 3, 6, 8, 7168, 1, 1, 0, "bf16"),
    (2, 2, 2, 4, 16400, 0, 1, 0, "f16"),
    (2, 3, 17, 24, 300, 0, 1, 0, "bf16"),
    (2, 400, 3, 4, 24, 0, 1, 2, "f16"),
    (2, 3, 4, 8, 2044, 0, 1, 0, "bf16"),
    (2, 3, 4, 8, 2046, 1, 0, 2, "f16"),
    (2, 3, 9, 16, 2047, 0, 1, 2, "bf16"),
    (2, 2, 2, 4, 9001, 0, 1, 0, "f16"),
]
ids_of = lambda c: "-".join(map(str, c))  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=ids_of)
def test_combine_backward(case):
    r = Routed(*case, seed=sum(case[:5]))
    g, g64 = r.rows((r.W, r.bs, r.h))
    y, y64 = r.expert_rows()
    got = r.combine_backward(g, y, x=True)
    r.check_combine(got, g64, y64)
    # the same bytes by a map rebuilt in another workspace, and each output by itself
    again = r.combine_backward(g, y, x=True, ws=M.alloc_workspace(r.cfg))
    only = [r.combine_backward(g, None, weights=False, x_in=False)["rows"], r.combine_backward(g, y, rows=False)["weights"],
            r.combine_backward(g, None, rows=False, weights=False, x=True, x_in=False)["x"]]
    for name, alone in zip(("rows", "weights", "x"), only):
        assert torch.equal(got[name], again[name]) and torch.equal(got[name], alone)


@pytest.mark.parametrize("case", CASES, ids=ids_of)
def test_dispatch_backward(case):
    r = Routed(*case, seed=sum(case[:5]) + 1)
    y, y64 = r.expert_rows()
    res, res64 = r.rows((r.W, r.bs, r.h))
    rw = torch.randn(r.W, r.A, device="cuda")
    r.check_dispatch(r.dispatch_backward(y), y64)
    got = r.dispatch_backward(y, res, rw)
    r.check_dispatch(got, y64, res64, rw)
    other = r.dispatch_backward(y, res, rw, ws=M.alloc_workspace(r.cfg))
    assert torch.equal(got[0], other[0]) and torch.equal(got[1], other[1])
    assert torch.equal(got[0], r.dispatch_backward(y, res.clone(), in_place=True)[0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_backward_against_differences(dtype):
    """Small whole numbers and weights of powers of two: combine and dispatch are exact, and linear in each of
    their inputs, so that a difference of the loss <c, output> is the gradient's product to the last bit."""
    r = Routed(2, 6, 3, 6, 24, 1, 2, 2, dtype, seed=3)
    whole = lambda *shape: torch.from_numpy(r.rng.integers(-2, 3, shape).astype(np.float32)).to(DT[dtype]).cuda()  # noqa: E731
    r.weights_d = torch.from_numpy(2.0 ** r.rng.integers(-1, 2, (r.W, r.bs, r.K)).astype(np.float32)).cuda()
    r.x = whole(r.W, r.bs, r.h)
    y, g = whole(r.W, r.A, r.h), whole(r.W, r.bs, r.h)

    def loss(y, w, x):
        out = torch.empty_like(x)
        M.combine(r.cfg, y, r.out["assist_info"], r.out["ep_recv_count"], r.ids_d, w, r.mask, x, out, None, r.ws)
        return float((out.double() * g.double()).sum())

    got = r.combine_backward(g, y, x=True)
    base = loss(y, r.weights_d, r.x)
    dy, dw, dx = whole(r.W, r.A, r.h), torch.randint(-2, 3, r.weights.shape, device="cuda").float(), whole(r.W, r.bs, r.h)
    there = torch.arange(r.A, device="cuda") < r.out["ep_recv_count"][:, -1:]
    assert loss(y + dy, r.weights_d, r.x) - base == float((got["rows"].double() * dy.double())[there].sum())
    assert loss(y, r.weights_d + dw, r.x) - base == float((got["weights"].double() * dw.double()).sum())
    assert loss(y, r.weights_d, r.x + dx) - base == float((got["x"].double() * dx.double()).sum())

    c, cw = whole(r.W, r.A, r.h), torch.randint(-2, 3, (r.W, r.A), device="cuda").float()

    def sent(x, w):
        out = M.alloc_dispatch_outputs(r.cfg, DT[dtype])
        M.dispatch(r.cfg, x, r.ids_d, r.mask, w, out["expand_x"], None, out["assist_info"], out["ep_recv_count"],
                   out["expand_scales"], None, M.alloc_workspace(r.cfg))
        return float((out["expand_x"].double() * c.double())[there].sum() + (out["expand_scales"].double() * cw.double())[there].sum())

    gx, gw = r.dispatch_backward(c, None, cw)
    assert sent(r.x + dx, r.weights_d) - sent(r.x, r.weights_d) == float((gx.double() * dx.double()).sum())
    assert sent(r.x, r.weights_d + dw) - sent(r.x, r.weights_d) == float((gw.double() * dw.double()).sum())


def test_infinities_stay_with_their_token():
    """What tokens and rows without a part hold is not read; what one token's hold does not reach another."""
    r = Routed(2, 6, 3, 6, 64, 1, 1, 2, "bf16", seed=8)
    g, g64 = r.rows((2, 6, 64))
    y, y64 = r.expert_rows()
    assert (r.cls[0, 0] == CLASS_NONE).all()
    g[0, 0], r.x[0, 0] = float("nan"), float("nan")
    dead = [(s, t, k) for s in range(2) for t in range(6) for k in range(3) if r.cls[s, t, k] == CLASS_NONE]
    for at in dead:
        r.weights_d[at] = float("inf")
    got = r.combine_backward(g, y, x=True)
    g64[0, 0] = 0.0
    r.check_combine(got, g64, y64)
    d, row = r.where[next(k for k in r.where if k[:2] == (1, 2))]
    y[d, row] = float("inf")
    g[1, 3] = float("inf")
    one = r.combine_backward(g, y, x=True)
    same = torch.ones(2, 6, dtype=torch.bool, device="cuda")
    same[1, 2] = same[1, 3] = False
    assert torch.equal(one["weights"][same], got["weights"][same]) and torch.equal(one["x"][same], got["x"][same])


@pytest.mark.parametrize("which", ["combine", "dispatch"])
def test_backward_reports_rows_that_do_not_match(which):
    def status(change):
        r = Routed(2, 6, 2, 4, 64, seed=5)
        r.ws = M.alloc_workspace(r.cfg)  # the map is rebuilt from what the arrays say
        change(r)
        y, g = torch.zeros(2, r.A, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 6, 64, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(y)
        if which == "combine":
            M.combine_backward(r.cfg, g, y, *r.route(), r.weights_d, None, None, out, ws=r.ws)
        else:
            M.dispatch_backward(r.cfg, y, *r.route(), None, g, ws=r.ws)
        return M.STATUS[M.get_device_status(r.ws)]

    assert status(lambda r: None) == "OK"
    assert status(lambda r: r.out["assist_info"][0, 1].fill_(-1)) == "BAD_ASSIST"
    assert status(lambda r: r.out["ep_recv_count"][1, -1:].sub_(1)) == "BAD_ASSIST"
    assert status(lambda r: r.out["ep_recv_count"][1, -1:].fill_(r.A + 1)) == "BAD_ASSIST"
    assert status(lambda r: r.ids_d[1, 2, 0].fill_(4)) == "BAD_EXPERT_ID"
    assert status(lambda r: r.ids_d[1, 2].copy_(r.ids_d[1, 2].flip(0))) == "BAD_ASSIST"


def test_backward_from_a_graph_and_on_a_side_stream():
    r = Routed(4, 16, 4, 16, 512, 1, 1, 2, "bf16", seed=6)
    g, _ = r.rows((4, 16, 512))
    y, _ = r.expert_rows()
    want = r.combine_backward(g, y, x=True)
    gx = r.dispatch_backward(y, g)[0]
    side = torch.cuda.Stream()
    other = r.combine_backward(g, y, x=True, stream=side)
    assert all(torch.equal(want[n], other[n]) for n in want)
    rows, weights, x, sums = (torch.full_like(t, 7.0) for t in (*want.values(), gx))
    graph = torch.cuda.CUDAGraph()
    ws = M.alloc_workspace(r.cfg)  # one workspace for the captured calls, another for those beside them
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        M.combine_backward(r.cfg, g, y, *r.route(), r.weights_d, r.mask, r.x, rows, weights, x, ws)
        M.dispatch_backward(r.cfg, y, *r.route(), r.mask, sums, g, ws=ws)
    for _ in range(2):
        for t in (rows, weights, x, sums):
            t.fill_(7.0)
        graph.replay()
        r.combine_backward(g, y, x=True)
        torch.cuda.synchronize()
        assert M.get_device_status(ws) == 0
        assert torch.equal(rows, want["rows"]) and torch.equal(weights, want["weights"]) and torch.equal(x, want["x"])
        assert torch.equal(sums, gx)


def test_two_batches_of_one_workspace():
    """The map of the batch that was dispatched last is not taken for another one's."""
    a = Routed(2, 20, 3, 8, 128, seed=10)
    b = Routed(2, 20, 3, 8, 128, seed=11)
    y, y64 = a.expert_rows()
    g, g64 = a.rows((2, 20, 128))
    b.ws = a.ws
    for r in (b, a, b):
        M.dispatch(r.cfg, r.x, r.ids_d, None, r.weights_d, r.out["expand_x"], None, r.out["assist_info"], r.out["ep_recv_count"],
                   r.out["expand_scales"], None, r.ws)
    a.check_combine(a.combine_backward(g, y), g64, y64)
    a.check_dispatch(a.dispatch_backward(y), y64)
    y, y64 = b.expert_rows()
    b.check_combine(b.combine_backward(g, y), g64, y64)


@pytest.mark.parametrize("bs", [20, 90, 700])
def test_rows_in_another_order(bs):
    """Rows permuted within their segments, as combine takes them: found all the same, by each gradient and with a map."""
    r = Routed(2, bs, 2, 4, 32, 0, 1, 2, "bf16", seed=bs)
    y, y64 = r.expert_rows()
    g, g64 = r.rows((2, bs, 32))
    order = np.tile(np.arange(r.A), (2, 1))
    for d in range(2):
        edges = [0, *r.ep[d]]
        for lo, hi in zip(edges[:-1], edges[1:]):
            order[d, lo:hi] = lo + r.rng.permutation(hi - lo)
    r.assist = np.take_along_axis(r.assist, order[..., None], 1)
    r.out["assist_info"] = torch.from_numpy(r.assist).cuda()  # in a buffer of its own: no map is its
    r.where = {tuple(r.assist[d, i]): (d, i) for d in range(2) for i in range(r.ep[d, -1])}
    r.check_combine(r.combine_backward(g, y, x=True), g64, y64)
    got = r.dispatch_backward(y, g)
    r.check_dispatch(got, y64, g64)
    assert M.get_device_status(r.ws) == 0


def test_rows_beyond_32_bits():
    """Rows that begin behind 2^31 elements of their array: two ranks of 33000 tokens, each with room for all of them."""
    W, bs, h = 2, 33000, 16448
    cfg = M.config(W, bs, h, 1, 2, torch.bfloat16)
    ws, A = M.alloc_workspace(cfg), M.workspace_size(cfg)[1]
    assert W * A * h > 2 ** 31
    ids = torch.ones(W, bs, 1, dtype=torch.int32, device="cuda")  # all to the second rank
    assist = torch.full((W, A, 3), -1, dtype=torch.int32, device="cuda")
    assist[1, :, 0] = torch.arange(A, device="cuda") // bs
    assist[1, :, 1] = torch.arange(A, device="cuda") % bs
    assist[1, :, 2] = 0
    ep = torch.tensor([[0, 0], [bs, 2 * bs]], dtype=torch.int32, device="cuda")
    w = torch.full((W, bs, 1), 0.5, device="cuda")
    g = torch.empty(W, bs, h, dtype=torch.bfloat16, device="cuda")
    g[:] = (torch.arange(W * bs, device="cuda") % 251 - 125).view(W, bs, 1)
    rows, gw = torch.zeros(W, A, h, dtype=torch.bfloat16, device="cuda"), torch.empty(W, bs, 1, device="cuda")
    rows[1] = 1.0
    y = rows.clone()
    M.combine_backward(cfg, g, y, assist, ep, ids, w, None, None, rows, gw, ws=ws)
    assert torch.equal(rows[1].view(W, bs, h), g * 0.5) and not bool(rows[0].any())
    assert torch.equal(gw.view(-1), g[..., 0].float().view(-1) * h)  # below 2^24: exact
    gx = torch.empty_like(g)
    M.dispatch_backward(cfg, rows, assist, ep, ids, None, gx, residual=g, ws=ws)
    assert torch.equal(gx, (g.float() * 1.5).bfloat16()) and M.get_device_status(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_training_step(dtype):
    """route -> dispatch -> experts -> combine forward, and back by the library's gradients, against the chain rule in
    64 bits on the same rounded intermediates."""
    W, bs, K, E, h = 4, 10, 3, 8, 96
    rng = np.random.default_rng(21)
    T = W * bs
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    cfg, rc = M.config(W, bs, h, K, E, DT[dtype]), M.router_config(T, E, K, torch.float32)
    ws, out = M.alloc_workspace(cfg), M.alloc_dispatch_outputs(cfg, DT[dtype])
    ids, weights = torch.empty(W, bs, K, dtype=torch.int32, device="cuda"), torch.empty(W, bs, K, device="cuda")
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DT[dtype]).cuda()  # noqa: E731
    x, g, gains = draw(W, bs, h), draw(W, bs, h), draw(E, h)  # an expert scales its rows by its gains
    M.route(rc, logits, None, ids, weights)
    M.dispatch(cfg, x, ids, None, weights, out["expand_x"], None, out["assist_info"], out["ep_recv_count"], None, None, ws)
    ep = out["ep_recv_count"]
    L, A = E // W, out["expand_x"].shape[1]
    at = torch.arange(A, device="cuda")
    expert = torch.stack([(at[:, None] >= ep[d].view(L, W)[:, -1]).sum(-1).clamp(max=L - 1) + d * L for d in range(W)])
    there = at < ep[:, -1:]
    y = torch.where(there[..., None], out["expand_x"], 0) * gains[expert]
    result = torch.empty_like(x)
    M.combine(cfg, y, out["assist_info"], ep, ids, weights, None, x, result, None, ws)
    # back
    gy, gw, gx, gl = torch.zeros_like(y), torch.empty_like(weights), torch.empty_like(x), torch.empty_like(logits)
    M.combine_backward(cfg, g, y, out["assist_info"], ep, ids, weights, None, None, gy, gw, ws=ws)
    grad_rows = gy * gains[expert]
    grad_gains = torch.zeros(E, h, dtype=torch.float64, device="cuda").index_add_(
        0, expert[there], (gy.double() * out["expand_x"].double())[there])
    M.dispatch_backward(cfg, grad_rows, out["assist_info"], ep, ids, None, gx, residual=g, ws=ws)
    M.route_backward(rc, logits, ids, gw, gl)
    assert M.get_device_status(ws) == 0

    # the chain rule, the choice of experts held fixed, with the way past the layer
    half = HALF_ULP[dtype]
    x64 = x.double().requires_grad_(True)
    l64 = logits.double().requires_grad_(True)
    g64 = gains.double().requires_grad_(True)
    pick = ids.long().view(T, K)
    share = torch.softmax(l64, -1).gather(1, pick)
    share = share / share.sum(-1, keepdim=True)
    xt = x64.view(T, h)
    by_pick = xt[:, None] * g64[pick]
    layer = (share[..., None] * by_pick).sum(1)
    ((layer + xt) * g.double().view(T, h)).sum().backward()
    size = (share[..., None] * by_pick).abs().sum(1).detach()
    # y is rounded once and its sum, of fp32 weights, once more
    off = (result.double().view(T, h) - layer.detach()).abs()
    assert bool((off <= half * layer.detach().abs() + (half + 64 * EPS) * size + TINY[dtype]).all())
    # w g and its product with the gains are rounded, then the sum
    parts = (share[..., None] * g.double().view(T, 1, h) * g64[pick]).abs().sum(1).detach()
    want = x64.grad.view(T, h)
    assert bool(((gx.double().view(T, h) - want).abs() <= half * want.abs() + (2 * half + 64 * EPS) * parts * (1 + half)
                 + 8 * EPS * g.double().view(T, h).abs() + 8 * TINY[dtype]).all())
    # the weights' gradient is of rounded y: <g, y> is off by half |g y|, and the logits' by r (d_k - sum d_j r_j)
    dots = (g.double().view(T, 1, h) * by_pick).abs().sum(-1).detach()
    off_w = (half + 64 * EPS) * dots
    tol = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(
        1, pick, share.detach() * (off_w + (off_w * share.detach()).sum(-1, keepdim=True))
        + 64 * EPS * share.detach() * (dots + dots.amax(-1, keepdim=True)))
    # (the 64-bit chain goes through a softmax over all experts, whose terms cancel: 2^-53 of each, some tens of times)
    assert bool(((gl.double() - l64.grad).abs() <= tol + 2.0 ** -44 * dots.amax()).all())
    # the gains' gradient, summed in 64 bits here, of w g rounded once
    sums = torch.zeros(E, h, dtype=torch.float64, device="cuda").index_add_(
        0, pick.reshape(-1), (share[..., None] * g.double().view(T, 1, h) * x64.view(T, 1, h)).abs().detach().view(-1, h))
    assert bool(((grad_gains - g64.grad).abs() <= (half + 64 * EPS) * sums + 1e-6 * (dtype == "f16")).all())
