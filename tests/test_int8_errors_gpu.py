"""The int8 product where something is wrong: what it writes for the experts whose counts are right when others' are
not, and a wait that runs out."""
import numpy as np
import pytest
import torch

from test_int8_gpu import DT, HALF_ULP, Product

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import moe as M

W, BS, TOPK, N = 2, 40, 2, 64
COUNTS = [3, 37, 20, 6, 0, 33]  # of three experts on each of two ranks

# what of the counts is changed (rank, local expert's end; its new value from the old counts and the capacity)
CHANGES = {
    "last end above the capacity": lambda ep, A: {(1, 2): A + 1},
    "an end above the capacity": lambda ep, A: {(0, 1): A + 7},
    "first end negative": lambda ep, A: {(0, 0): -1},
    "decreasing": lambda ep, A: {(0, 2): ep(0, 1) - 1},
    "smallest number": lambda ep, A: {(1, 1): -2 ** 31},
    "largest number": lambda ep, A: {(0, 2): 2 ** 31 - 1},
    "both ranks": lambda ep, A: {(0, 2): A + 1, (1, 0): -5},
    "an expert has its neighbour's rows and more": lambda ep, A: {(0, 1): ep(0, 2) + 2},
}


@pytest.mark.parametrize("k", [64, 65, 400])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("change", CHANGES, ids=lambda c: c.replace(" ", "_").replace("'", ""))
def test_experts_beside_one_of_wrong_counts(change, swiglu, k):
    """Of an expert's counts its rows' begin and end are read. Where they are wrong its rows are passed over, and all
    others are computed as their own counts say."""
    pr = Product(W, BS, TOPK, COUNTS, N, k, seed=k)
    L = len(COUNTS) // W
    ep = pr.ep.copy()
    at = lambda d, le: (d, le * W + W - 1)  # noqa: E731
    for (d, le), v in CHANGES[change](lambda d, le: int(pr.ep[at(d, le)]), pr.A).items():
        ep[at(d, le)] = v
    y = pr.run("bf16", swiglu, expect="BAD_ASSIST", ep=ep)
    got = y.double().cpu().numpy()
    written = np.zeros((W, pr.A), dtype=bool)
    good = 0
    for e in range(len(COUNTS)):
        d, le = divmod(e, L)
        lo, hi = int(ep[at(d, le - 1)]) if le else 0, int(ep[at(d, le)])
        if not 0 <= lo <= hi <= pr.A:
            continue
        good += 1
        assert not written[d, lo:hi].any()  # (the changes leave no row to two good experts)
        written[d, lo:hi] = True
        pr.ranges[e] = (d, lo, hi)
        want, tol = pr.want(e, swiglu)
        off = np.abs(got[d, lo:hi] - want) - (tol + HALF_ULP["bf16"] * (np.abs(want) + tol) + 1e-40)
        assert (off <= 0).all(), e
    assert good < len(COUNTS)
    assert bool((y[torch.from_numpy(~written).cuda()] == 777.0).all())  # (776 in bf16, as it was filled)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """Rows of 131056 elements take a unit's MMAs some hundred microseconds, so that the epilogue's wait for them lasts
    longer than a limit of one: the call ends, says so, and leaves the device usable. Two to three units a pair of CTAs:
    copies, widening, MMAs and epilogue all meet the abort."""
    k, n, E = 131056, 256 * 50, 4
    cfg = M.config(2, 2, 64, 2, E, torch.bfloat16, quant_mode=2)
    ws, A = M.alloc_workspace(cfg), M.workspace_size(cfg)[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-127, 128, (2, A, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.zeros(E, n, k, dtype=torch.int8, device="cuda")
    w[:, :, :256] = torch.randint(-127, 128, (E, n, 256), generator=g, device="cuda", dtype=torch.int8)
    xs, wsc = torch.rand(2, A, generator=g, device="cuda") + 0.5, (torch.rand(E, n, generator=g, device="cuda") + 0.5) / 4096
    ep = torch.tensor([[1, 1, 2, 2], [1, 1, 2, 2]], dtype=torch.int32, device="cuda")  # a row for each expert
    y = torch.full((2, A, n), 777.0, dtype=torch.bfloat16, device="cuda")

    def call(limit_us):
        cfg.wait_timeout_us = limit_us
        M.expert_product_int8(cfg, x, xs, ep, w, wsc, y, ws=ws)
        return M.STATUS[M.get_device_status(ws)]

    limit = cfg.wait_timeout_us
    assert call(1) == "TIMEOUT"
    y.fill_(777.0)
    assert call(limit) == "OK"
    rows = x[:, :2, :256].double().reshape(E, 1, 256)  # rank d's row le is its local expert le's
    want = (rows @ w[:, :, :256].double().transpose(1, 2))[:, 0] * xs[:, :2].double().reshape(E, 1) * wsc.double()
    got = y[:, :2].double().reshape(E, n)
    # whole sums below 2^24, two products with the scales, and the rounding to 16 bits
    tol = 3 * 2.0 ** -24 * want.abs()
    assert bool(((got - want).abs() <= tol + HALF_ULP["bf16"] * (want.abs() + tol) + 1e-40).all())
    assert bool((y[:, 2:] == 777.0).all())
