"""Operators around the experts (include/moe_experts.h) at layouts and counts
beside the usual ones: rows of logits and gradients aligned differently, batches
of many experts, receive counts that are wrong in one place."""
import itertools

import numpy as np
import pytest
import torch

import experts_plain as P
from test_experts_gpu import DT, EPS, HALF_ULP, Product, product_want, rounded, run_product

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()


# ------------------------------------------------------------------ the router's gradient

def laid_out(T, E, dtype, pad, offset, fill):
    """A [T, E] view whose rows are E + pad elements apart and begin `offset` elements behind an
    allocation's start, and the whole of what it lies in."""
    whole = torch.full((T * (E + pad) + offset,), fill, dtype=dtype, device="cuda")
    return whole[offset:].view(T, E + pad)[:, :E], whole


def gradient(x, ids, grad, sigmoid, renorm, scaling, dtype, logits_at, grad_at):
    T, E = x.shape
    logits, _ = laid_out(T, E, dtype, *logits_at, float("nan"))
    logits.copy_(torch.from_numpy(x))
    out, whole = laid_out(T, E, dtype, *grad_at, 7.0)
    rc = M.router_config(T, E, ids.shape[1], dtype, score_func=int(sigmoid), renormalize=renorm, scaling=scaling,
                         logits_stride=E + logits_at[0])
    M.route_backward(rc, logits, torch.from_numpy(ids).cuda(), torch.from_numpy(grad).cuda(), out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    out.fill_(7.0)
    assert bool((whole == 7.0).all())  # nothing was written beside the rows
    return got


def check_gradient(T, E, K, dt, sigmoid, renorm, logits_at, grad_at, tokens):
    rng = np.random.default_rng(T + E + K)
    x = rounded(rng.standard_normal((T, E)) * 2, DT[dt])
    x[T // 2, rng.permutation(E)[: E // 4]] = -np.inf
    ids = np.argsort(-x, axis=1, kind="stable")[:, :K].astype(np.int32)
    grad = rng.standard_normal((T, K)).astype(np.float32)
    got = gradient(x, ids, grad, sigmoid, renorm, 2.5, DT[dt], logits_at, grad_at)
    for t in tokens:
        want = P.route_gradient(x[t], ids[t], grad[t], sigmoid, renorm, 2.5)
        # as in test_route_backward: terms of size share * (|g| + |mean|), exponentials of rounded
        # differences, sums of E / 32 (E / 16 of two tokens a warp) and five numbers; the type's own rounding
        s = P.scores(x[t], sigmoid)[0]
        share = s / (s[ids[t]].sum() if renorm else 1.0)
        fin = x[t][np.isfinite(x[t])]
        tol = (2 * (fin.max() - fin.min()) + E / 16 + 48) * EPS * 2.5 * np.abs(grad[t]).max() * 2
        assert (np.abs(got[t] - want) <= tol * share + HALF_ULP[dt] * np.abs(want) + 1e-7 * (dt == "f16") + 1e-30).all(), t


# (pad, offset) of the logits and of the gradient, in elements
LAYOUTS = [((0, 0), (1, 0)), ((1, 0), (0, 0)), ((0, 1), (0, 0)), ((0, 0), (0, 1)), ((32, 0), (0, 0)), ((1, 0), (3, 1))]


@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("logits_at,grad_at", LAYOUTS)
def test_gradient_rows_aligned_unlike_the_logits(logits_at, grad_at, E, dt, sigmoid, renorm):
    check_gradient(5, E, 6, dt, sigmoid, renorm, logits_at, grad_at, range(5))


@pytest.mark.parametrize("sigmoid,renorm", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("E,dt", [(256, "f32"), (128, "bf16")])
@pytest.mark.parametrize("logits_at,grad_at", LAYOUTS[:4])
def test_gradient_of_large_batches_aligned_unlike_the_logits(logits_at, grad_at, E, dt, sigmoid, renorm):
    """Beyond the batches from which two tokens share a warp where both sides are aligned."""
    T = 16387
    check_gradient(T, E, 8, dt, sigmoid, renorm, logits_at, grad_at, [*range(20), *range(T // 2 - 5, T // 2 + 5), *range(T - 20, T)])


# ------------------------------------------------------------------ the quantiser's layouts

def test_quantiser_refuses_layouts_that_there_are_not():
    """One beyond 32 bits is not cut to one that there is."""
    x = torch.randn(4, 64, device="cuda")
    codes, scales = M.alloc_mx(x, M.SF_TILED)
    for layout in (1 << 32, (1 << 32) + 1, -(1 << 32)):
        with pytest.raises(ValueError, match="layout"):
            M.mx_quantize(x, codes, scales, layout)
    for layout in (2, -1):
        with pytest.raises(M.MoeError, match="INVALID_ARG"):
            M.mx_quantize(x, codes, scales, layout)


# ------------------------------------------------------------------ the product's receive counts

def check_experts(pr, y, swiglu, dt, refused=()):
    """The refused experts' rows, and those beyond the counts, hold what they held; the others the product."""
    fill = torch.ones(pr.W, pr.A, dtype=torch.bool)
    for e, (d, lo, hi) in enumerate(pr.ranges):
        if e in refused or hi == lo:
            continue
        fill[d, lo:hi] = False
        want, tol = product_want(pr, e, swiglu)
        got = y[d, lo:hi].double().cpu().numpy()
        assert (np.abs(got - want) <= tol + HALF_ULP[dt] * (np.abs(want) + tol) + 1e-40).all(), e
    assert bool((y.cpu()[fill] == 777.0).all())


@pytest.mark.parametrize("bad,refused", [("above", (3,)), ("above inside", (0, 1)), ("negative", (0, 1)), ("decreasing", (1,))])
def test_product_leaves_out_the_experts_of_bad_counts_alone(bad, refused):
    pr = Product(2, 8, 2, [3, 4, 5, 6], 64, 64, seed=2)
    ep = pr.ep.copy()  # [rank][expert, source]: an expert's end is its second entry
    if bad == "above":
        ep[1, 3] = pr.A + 1
    elif bad == "above inside":
        ep[0, 1] = pr.A + 1
    elif bad == "negative":
        ep[0, 1] = -1
    else:
        ep[0, 3] = ep[0, 1] - 1
    y, _ = run_product(pr, "bf16", False, expect="BAD_ASSIST", ep=ep)
    check_experts(pr, y, False, "bf16", refused)


def test_product_reads_the_counts_at_the_experts_ends_alone():
    pr = Product(4, 8, 2, [3, 4, 5, 6, 0, 16, 1, 2], 64, 64, seed=6)
    ep = pr.ep.copy()
    ep.reshape(4, 2, 4)[..., :3] = np.array([-5, 1 << 30, 7])
    y, _ = run_product(pr, "bf16", False, ep=ep)
    check_experts(pr, y, False, "bf16")


@pytest.mark.parametrize("E,swiglu", [(450, False), (512, True), (1024, False)])
def test_product_of_more_experts_than_threads(E, swiglu):
    """Their running row tiles take more than one pass of a CTA's 448 threads; rows on either side of its end."""
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 4, E)
    counts[[0, 446, 447, 448, E - 1]] = 131, 5, 130, 3, 129
    pr = Product(2, 300, 2, counts.tolist(), 66, 96, seed=E)
    y, _ = run_product(pr, "bf16", swiglu)
    check_experts(pr, y, swiglu, "bf16")


# ------------------------------------------------------------------ scores of small size

def far_below(rng, T, E, K, G, KG):
    """fp32 logits whose sigmoid scores are all below 2^-28, those that the choice hangs on 2^-15 of their
    size apart: twice what two keys are off."""
    out = np.empty((T, E))
    for t in range(T):
        while True:
            x = rounded(np.clip(rng.standard_normal(E) * 6 - 50, -80, -20), torch.float32)
            _, key = P.keys(x, None, True, True)
            v = P.group_values(key, G, True)
            opened = sorted(range(G), key=lambda g: (-v[g], g))[:KG]
            left = np.sort(key[np.isin(np.arange(E) // (E // G), opened)])[::-1][: K + 1]
            ordered = np.sort(v)[::-1]
            if all(((a[:-1] - a[1:]) > 2.0 ** -15 * a[:-1]).all() for a in (left, ordered)):
                break
        out[t] = x
    return out


@pytest.mark.parametrize("T,E,K,G,KG", [(40, 64, 6, 4, 2), (40, 256, 8, 8, 4), (40, 60, 5, 6, 3), (8195, 256, 8, 8, 4), (8195, 128, 4, 2, 1)])
def test_route_by_scores_far_below_one(T, E, K, G, KG):
    """Keys of scores alone order by their own size, not by how near to one another they are."""
    rng = np.random.default_rng(E + T)
    some = far_below(rng, min(T, 64), E, K, G, KG)
    x = some[np.arange(T) % len(some)]
    logits = torch.from_numpy(x).float().cuda()
    rc = M.router_config(T, E, K, torch.float32, G, KG, M.GROUP_TOP2_SUM, M.SCORE_SIGMOID, True, 1.0)
    ids = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    M.route(rc, logits, None, ids, w)
    want = [P.route_token(r, None, K, G, KG, True, True, True, 1.0) for r in some]
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    for t in range(T):
        ri, rw = want[t % len(some)]
        assert np.array_equal(ids[t], ri), t
        assert (np.abs(w[t] - rw) <= 64 * EPS * rw).all(), t  # exponentials, a sum and a division of some ulps each


@pytest.mark.parametrize("T", [3, 8193])
def test_renormalised_weights_and_gradient_of_scores_below_fp32(T):
    """Sigmoid scores of logits under -88 are 0 in fp32: the picks go by the logits, their weights and gradients are 0."""
    x = -95.0 - torch.arange(128, device="cuda").flip(0).float()[None] / 8 + torch.zeros(T, 1, device="cuda")
    rc = M.router_config(T, 128, 4, torch.float32, score_func=M.SCORE_SIGMOID)
    ids, w = torch.zeros(T, 4, dtype=torch.int32, device="cuda"), torch.full((T, 4), float("nan"), device="cuda")
    M.route(rc, x, None, ids, w)
    assert bool((ids == torch.tensor([127, 126, 125, 124], device="cuda")).all()) and bool((w == 0).all())
    g = torch.full_like(x, 7.0)
    M.route_backward(rc, x, ids, torch.ones_like(w), g)
    assert bool((g == 0).all())
