"""The operators around the experts (include/moe_experts.h) through the C ABI
against their plain 64-bit forms (experts_plain.py): routing and its gradient,
MX FP4 quantisation, and the grouped product."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import experts_plain as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()

EPS = 2.0 ** -24  # half an ulp of 1 in fp32
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": EPS, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # relative, one rounding


def strided(a, dtype, pad):
    """A CUDA copy of a 2D array whose rows are `pad` elements further apart than they are long."""
    t = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, : a.shape[1]] = torch.from_numpy(a).to(dtype).cuda()
    return t[:, : a.shape[1]]


def rounded(a, dtype):
    """The numbers that an array holds after rounding to dtype."""
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dtype).double().numpy()


# ------------------------------------------------------------------ routing

def separated_logits(rng, T, E, dtype, bias, sigmoid, K, G, KG, top2, masked=0):
    """Logits (as dtype holds them) whose choice does not hang on fp32 rounding: where keys
    are scores, those that are chosen or next to it, and the groups' values, are equal or
    2^-17 of their size apart (a score is within (|x - top| + E / 32 + some) * 2^-24)."""
    def apart(a):
        a = a[a != -np.inf]
        gap = a[:-1] - a[1:]
        return ((gap == 0) | (gap > 2.0 ** -17 * np.maximum(np.abs(a[:-1]), np.abs(a[1:])))).all()

    out = np.empty((T, E))
    for t in range(T):
        for _ in range(500):
            x = rounded(rng.standard_normal(E) * 2, dtype)
            x[rng.permutation(E)[:masked]] = -np.inf
            if bias is None and not top2:
                break
            _, key = P.keys(x, bias, sigmoid, top2)
            v = P.group_values(key, G, top2)
            opened = sorted(range(G), key=lambda g: (-v[g], g))[:KG]
            left = np.sort(key[np.isin(np.arange(E) // (E // G), opened)])[::-1]
            if apart(left[: K + 1]) and apart(np.sort(v)[::-1]):
                break
        else:
            raise AssertionError("no separated logits found")
        out[t] = x
    return out


def run_route(x, bias, K, G, KG, sigmoid, top2, renorm, scaling, dtype, pad=0, stream=None):
    T, E = x.shape
    logits = strided(x, dtype, pad) if pad else torch.from_numpy(x).to(dtype).cuda()
    rc = M.router_config(T, E, K, dtype, G, KG, M.GROUP_TOP2_SUM if top2 else M.GROUP_MAX,
                         M.SCORE_SIGMOID if sigmoid else M.SCORE_SOFTMAX, renorm, scaling, E + pad)
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).cuda()
    M.route(rc, logits, b, ids, w, stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check_route(x, bias, K, G, KG, sigmoid, top2, renorm, scaling, dtype, pad=0):
    ids, w = run_route(x, bias, K, G, KG, sigmoid, top2, renorm, scaling, dtype, pad)
    for t in range(x.shape[0]):
        ri, rw = P.route_token(x[t], bias, K, G, KG, sigmoid, top2 and G > 1, renorm, scaling)
        assert np.array_equal(ids[t], ri), (t, ids[t], ri, x[t])
        # exp's argument is rounded (relative error |x - top| * EPS of the exponential), its value and the
        # division by some ulps each, a sum of up to E positive terms by E / 32 + 5 additions, the sum over picks by 5
        fin = x[t][np.isfinite(x[t])]
        span = float(fin.max() - fin.min()) if fin.size and not sigmoid else 0.0
        tol = (2 * min(span, 200.0) + x.shape[1] / 32 + 32) * EPS
        assert (np.abs(w[t] - rw) <= tol * np.abs(rw) + 1e-37).all(), (t, w[t], rw)


ROUTE_CASES = [
    # T, E, K, G, KG, sigmoid, top2, bias, renorm, dtype, pad, masked
    (1, 256, 8, 8, 4, True, True, True, True, "f32", 0, 0),
    (3, 256, 8, 8, 4, True, True, True, False, "f32", 0, 30),
    (37, 128, 8, 1, 1, False, False, False, True, "bf16", 0, 0),
    (5, 128, 6, 1, 1, False, False, False, False, "f16", 8, 5),
    (9, 64, 4, 4, 2, False, False, True, True, "f32", 3, 0),
    (7, 60, 5, 6, 3, True, True, True, True, "bf16", 1, 7),
    (4, 1, 1, 1, 1, False, False, False, True, "f32", 0, 0),
    (4, 7, 7, 1, 1, False, False, False, True, "f32", 0, 2),
    (6, 33, 32, 1, 1, True, False, True, True, "f32", 0, 0),
    (3, 1024, 32, 1, 1, False, False, False, True, "bf16", 0, 0),
    (3, 1024, 32, 32, 8, True, True, True, True, "f32", 0, 100),
    (5, 1023, 17, 3, 1, False, True, False, False, "f16", 5, 0),
    (8, 96, 8, 8, 3, False, False, False, True, "bf16", 0, 0),
    (8, 160, 6, 8, 3, False, False, False, False, "bf16", 0, 0),
    (4, 16, 4, 16, 4, True, True, True, True, "f32", 0, 0),
    (5, 512, 10, 1, 1, False, False, True, True, "f32", 0, 0),
    (5, 384, 8, 1, 1, True, False, True, True, "f32", 0, 0),
    (130, 256, 1, 8, 1, True, True, True, False, "bf16", 0, 0),
    (2, 64, 8, 8, 1, True, True, True, True, "f32", 0, 60),
    (2, 256, 16, 2, 2, True, True, False, True, "f32", 0, 0),
    (3, 512, 9, 8, 2, False, False, True, True, "bf16", 8, 9),
]


@pytest.mark.parametrize("case", ROUTE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_route(case):
    T, E, K, G, KG, sigmoid, top2, with_bias, renorm, dt, pad, masked = case
    rng = np.random.default_rng(sum(int(v) for v in case if not isinstance(v, str)) + E)
    bias = np.round(rng.uniform(-0.1, 0.1, E), 3).astype(np.float32) if with_bias else None
    x = separated_logits(rng, T, E, DT[dt], bias, sigmoid, K, G, KG, top2 and G > 1, masked)
    check_route(x, bias, K, G, KG, sigmoid, top2, renorm, 2.5, DT[dt], pad)


ROUTE_LARGE_CASES = [
    # E, K, G, KG, sigmoid, top2, bias, renorm, dtype
    (256, 8, 8, 4, True, True, True, True, "f32"), (256, 16, 1, 1, False, False, False, True, "bf16"),
    (128, 8, 1, 1, False, False, False, True, "bf16"), (128, 6, 4, 2, False, False, True, False, "f16"),
    (64, 6, 1, 1, True, False, True, True, "f32"), (64, 4, 16, 4, True, True, False, False, "bf16"),
    (256, 2, 2, 1, False, True, False, True, "f16"), (60, 4, 1, 1, False, False, False, True, "f32")]


def check_large_batch(case, T):
    E, K, G, KG, sigmoid, top2, with_bias, renorm, dt = case
    rng = np.random.default_rng(E + K)
    bias = np.round(rng.uniform(-0.1, 0.1, E), 3).astype(np.float32) if with_bias else None
    some = separated_logits(rng, 48, E, DT[dt], bias, sigmoid, K, G, KG, top2 and G > 1, masked=E // 16)
    x = some[rng.integers(0, len(some), T)]  # the checked tokens at any place of a warp
    x[-1] = some[0]
    if not with_bias and not top2:
        x[1::7] = rounded(rng.integers(-2, 3, x[1::7].shape) * 0.5, DT[dt])  # many equal keys
        x[5::64] = -np.inf
    ids, w = run_route(x, bias, K, G, KG, sigmoid, top2, renorm, 2.5, DT[dt])
    want = {}
    for t in range(T):
        key = x[t].tobytes()
        if key not in want:
            want[key] = P.route_token(x[t], bias, K, G, KG, sigmoid, top2 and G > 1, renorm, 2.5)
        ri, rw = want[key]
        assert np.array_equal(ids[t], ri), (t, ids[t], ri)
        assert (np.abs(w[t] - rw) <= 128 * EPS * np.abs(rw) + 1e-37).all(), t  # spans of 20 and sums of 256 at most


@pytest.mark.parametrize("case", ROUTE_LARGE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_route_large_batches(case):
    check_large_batch(case, 4099)


@pytest.mark.parametrize("case", ROUTE_LARGE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_route_batches_of_two_tokens_a_warp(case):
    check_large_batch(case, 8195)  # an odd last token


@pytest.mark.parametrize("E,K,G,KG", [(64, 8, 1, 1), (256, 8, 8, 4), (100, 10, 5, 2), (1024, 32, 4, 2)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_route_ties_go_to_the_lowest_index(E, K, G, KG, dt):
    rng = np.random.default_rng(E)
    x = rng.integers(-2, 3, (17, E)).astype(np.float64) * 0.5
    x[0] = 0.0
    x[1] = np.where(rng.random(E) < 0.5, 0.0, -0.0)  # the two zeros are one key
    check_route(x, None, K, G, KG, False, False, True, 1.0, DT[dt])


@pytest.mark.parametrize("sigmoid,renorm,G", list(itertools.product((False, True), (False, True), (1, 4))))
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_route_masked_and_extreme_rows(sigmoid, renorm, G, dt):
    """Rows with nothing left, one expert left, NaN, infinities and the type's lowest value."""
    E, K = 32, 4
    lowest = float(torch.finfo(DT[dt]).min)
    rng = np.random.default_rng(3)
    x = np.tile(rounded(rng.standard_normal(E), DT[dt]), (9, 1))
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, 19] = 0.25
    x[3, ::2] = np.nan
    x[4] = lowest
    x[5, 3:] = lowest
    x[6, 5] = x[6, 9] = np.inf
    x[7, :] = -np.inf
    x[7, 30:] = 1.0
    x[8, 1::2] = -np.inf
    check_route(x, None, K, G, min(G, 2), sigmoid, False, renorm, 1.0, DT[dt])
    if not sigmoid:
        return
    bias = np.zeros(E, dtype=np.float32)
    bias[4] = -np.inf
    bias[6] = np.nan
    y = x[[0, 2, 8]]
    check_route(y, bias, K, G, min(G, 2), sigmoid, G > 1, renorm, 1.0, DT[dt])


def test_route_no_tokens_side_stream_and_graph():
    rc = M.router_config(0, 8, 2, torch.float32)
    empty = torch.empty(0, 8, device="cuda")
    M.route(rc, empty, None, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    rng = np.random.default_rng(5)
    x = rng.standard_normal((50, 64))
    want = run_route(x, None, 6, 1, 1, False, False, True, 1.0, torch.float32)
    side = torch.cuda.Stream()
    got = run_route(x, None, 6, 1, 1, False, False, True, 1.0, torch.float32, stream=side)
    assert all(np.array_equal(a, b) for a, b in zip(want, got))
    logits = torch.from_numpy(x).float().cuda()
    rc = M.router_config(50, 64, 6, torch.float32)
    ids = torch.zeros(50, 6, dtype=torch.int32, device="cuda")
    w = torch.zeros(50, 6, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.route(rc, logits, None, ids, w)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), want[0]) and np.array_equal(w.cpu().numpy().astype(np.float64), want[1])


def run_grad(x, ids, grad, sigmoid, renorm, scaling, dtype, pad=0):
    T, E = x.shape
    logits = strided(x, dtype, pad) if pad else torch.from_numpy(x).to(dtype).cuda()
    out = torch.full((T, E + pad), 7.0, dtype=dtype, device="cuda")
    rc = M.router_config(T, E, ids.shape[1], dtype, score_func=int(sigmoid), renormalize=renorm, scaling=scaling,
                         logits_stride=E + pad)
    view = out[:, :E] if pad else out
    M.route_backward(rc, logits, torch.from_numpy(ids).cuda(), torch.from_numpy(grad).float().cuda(), view)
    torch.cuda.synchronize()
    assert pad == 0 or bool((out[:, E:] == 7.0).all())  # the gaps between rows stay
    return view.double().cpu().numpy()


@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
@pytest.mark.parametrize("T,E,K,dt,pad", [(1, 256, 8, "f32", 0), (33, 128, 8, "bf16", 0), (5, 60, 3, "f16", 4),
                                          (3, 1024, 32, "f32", 0), (4, 1, 1, "f32", 0), (7, 37, 37 - 5, "bf16", 3),
                                          (6, 257, 2, "f32", 1), (2, 512, 16, "bf16", 8), (70, 64, 6, "f16", 0)])
def test_route_backward(sigmoid, renorm, T, E, K, dt, pad):
    rng = np.random.default_rng(T * E + K)
    x = rounded(rng.standard_normal((T, E)) * 2, DT[dt])
    if E > 8:
        x[T // 2, rng.permutation(E)[: E // 4]] = -np.inf
    ids = np.stack([P.route_token(r, None, K, 1, 1, sigmoid, False, renorm, 1.0)[0] for r in x])
    grad = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(x, ids, grad, sigmoid, renorm, 2.5, DT[dt], pad)
    for t in range(T):
        want = P.route_gradient(x[t], ids[t], grad[t], sigmoid, renorm, 2.5)
        # terms of size r * (|g| + |mean|), each a handful of roundings; the type's own rounding of the result
        size = 2.5 * (np.abs(grad[t]).max() * 2)
        fin = x[t][np.isfinite(x[t])]
        tol = (2 * (fin.max() - fin.min()) + E / 32 + 48) * EPS * size
        assert (np.abs(got[t] - want) <= tol * np.maximum(P.scores(x[t], sigmoid)[0], 1e-30) * (
            1.0 if not renorm else 1.0 / max(P.scores(x[t], sigmoid)[0][ids[t]].sum(), 1e-30)) + HALF_ULP[dt] * np.abs(want) + 1e-7 * (dt == "f16")).all(), t


@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
@pytest.mark.parametrize("E,K,dt", [(256, 8, "f32"), (256, 16, "bf16"), (128, 8, "f16"), (64, 6, "f32"), (128, 4, "bf16")])
def test_route_backward_large_batches(sigmoid, renorm, E, K, dt):
    check_large_gradient(sigmoid, renorm, E, K, dt, 4097)


@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
@pytest.mark.parametrize("E,K,dt", [(256, 8, "f32"), (256, 16, "bf16"), (256, 4, "f16"), (128, 8, "f32")])
def test_route_backward_larger_batches(sigmoid, renorm, E, K, dt):
    check_large_gradient(sigmoid, renorm, E, K, dt, 16387)


def check_large_gradient(sigmoid, renorm, E, K, dt, T):
    rng = np.random.default_rng(E + K)
    x = rounded(rng.standard_normal((T, E)) * 2, DT[dt])
    x[7::50, : E // 4] = -np.inf
    x[9] = -np.inf
    ids = np.argsort(-x, axis=1, kind="stable")[:, :K].astype(np.int32)
    grad = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(x, ids, grad, sigmoid, renorm, 1.5, DT[dt])
    for t in [*range(0, 40), *range(T - 40, T), *rng.integers(0, T, 60)]:
        want = P.route_gradient(x[t], ids[t], grad[t], sigmoid, renorm, 1.5)
        # probabilities and shares are at most 1; terms of size |g|, each some 64 roundings and spans of 20 at most
        assert np.allclose(got[t], want, rtol=HALF_ULP[dt], atol=128 * EPS * 3 * np.abs(grad[t]).max() + 6e-8 * (dt == "f16")), t


@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
def test_route_backward_against_differences(sigmoid, renorm):
    """Central differences of the 64-bit weights, the choice held fixed."""
    rng = np.random.default_rng(8)
    T, E, K, h = 3, 24, 5, 1e-5
    x = rounded(rng.standard_normal((T, E)), torch.float32)
    ids = np.stack([P.route_token(r, None, K, 1, 1, sigmoid, False, renorm, 1.0)[0] for r in x])
    grad = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(x, ids, grad, sigmoid, renorm, 1.5, torch.float32)
    for t, e in itertools.product(range(T), range(E)):
        up, down = x[t].copy(), x[t].copy()
        up[e] += h
        down[e] -= h
        diff = (P.weights_of(up, ids[t], sigmoid, renorm, 1.5) - P.weights_of(down, ids[t], sigmoid, renorm, 1.5)) @ grad[t] / (2 * h)
        # the differences' own error: h^2 / 6 of a third derivative of order one, and 1e-16 / h
        assert abs(got[t, e] - diff) <= 1e-5


def test_route_backward_masked_rows_and_foreign_ids():
    E, K = 40, 4
    x = np.full((4, E), -np.inf)
    x[1, 3] = 1.0
    x[2] = np.nan
    x[3] = 0.5
    ids = np.stack([P.route_token(r, None, K, 1, 1, False, False, True, 1.0)[0] for r in x])
    grad = np.ones((4, K), dtype=np.float32)
    for sigmoid, renorm in itertools.product((False, True), (False, True)):
        got = run_grad(x, ids, grad, sigmoid, renorm, 1.0, torch.float32)
        for t in range(4):
            want = P.route_gradient(x[t], ids[t], grad[t], sigmoid, renorm, 1.0)
            assert np.allclose(got[t], want, rtol=0, atol=64 * EPS), (sigmoid, renorm, t)
    odd = ids.copy()
    odd[3, 1], odd[3, 2] = -1, E  # passed over
    got = run_grad(x, odd, grad, True, False, 1.0, torch.float32)
    s = 1 / (1 + np.exp(-0.5))
    want = np.zeros(E)
    want[[odd[3, 0], odd[3, 3]]] = s * (1 - s)
    assert np.allclose(got[3], want, rtol=0, atol=8 * EPS)


@pytest.mark.parametrize("T,E", [(5, 40), (3, 128), (4160, 128)])
@pytest.mark.parametrize("sigmoid,renorm", list(itertools.product((False, True), (False, True))))
def test_route_backward_passes_over_gradients_of_masked_picks(sigmoid, renorm, T, E):
    """Infinities and NaN there (a loss of the weights' logarithms has them) reach no other expert."""
    rng = np.random.default_rng(21)
    K = 4
    x = np.full((T, E), -np.inf)
    x[:, 7:9] = rounded(rng.standard_normal((T, 2)), torch.float32)
    ids = np.tile(np.array([8, 0, 7, 1], dtype=np.int32), (T, 1))
    grad = rng.standard_normal((T, K)).astype(np.float32)
    clean = grad.copy()
    grad[:, 1], grad[:, 3] = np.inf, np.nan
    clean[:, [1, 3]] = 0
    got = run_grad(x, ids, grad, sigmoid, renorm, 1.5, torch.float32)
    for t in range(0, T, 1 + T // 64):
        want = P.route_gradient(x[t], ids[t], clean[t], sigmoid, renorm, 1.5)
        assert np.allclose(got[t], want, rtol=HALF_ULP["f32"], atol=128 * EPS * 3 * np.abs(clean[t]).max()), t
    assert np.isfinite(got).all() and (np.delete(got, [7, 8], 1) == 0).all()


# ------------------------------------------------------------------ MX FP4 quantisation

def run_quantize(x, dtype, layout, pad=0):
    E, rows, cols = x.shape
    t = torch.full((E, rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    t[..., :cols] = torch.from_numpy(x).to(dtype).cuda()
    t = t[..., :cols]
    codes, scales = M.alloc_mx(t, layout)
    codes.fill_(0xA5), scales.fill_(0xA5)
    M.mx_quantize(t, codes, scales, layout)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


def edge_values(rng, n, dtype):
    """Numbers around the format's rounding boundaries and over the type's range."""
    grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7, 7.75])
    v = rng.choice(grid, n) * np.exp2(rng.integers(-1, 1, n)) * rng.choice([-1, 1], n)
    step = np.where(rng.random(n) < 0.3, rng.choice([-1, 1], n) * 2.0 ** -10, 0.0)
    return rounded(v * (1 + step), dtype)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("E,rows,cols,dt,pad", [
    (1, 1, 32, "bf16", 0), (1, 5, 2, "f32", 0), (2, 3, 30, "f16", 2), (1, 130, 64, "bf16", 0), (3, 129, 96, "f32", 0),
    (2, 33, 34, "bf16", 6), (1, 7, 2048, "bf16", 0), (1, 3, 7168, "f16", 0), (2, 128, 128, "f32", 4), (1, 31, 1000, "bf16", 8),
    (1, 9, 480, "f16", 1), (4, 64, 256, "bf16", 0), (2, 257, 288, "bf16", 32)])
def test_quantize(layout, E, rows, cols, dt, pad):
    rng = np.random.default_rng(rows * cols + E)
    x = rounded(rng.standard_normal((E, rows, cols)), DT[dt])
    x[:, ::3] = edge_values(rng, x[:, ::3].size, DT[dt]).reshape(x[:, ::3].shape)
    x[:, 1::5] *= 2.0 ** -12
    x[0, 0, : min(32, cols)] = 0.0
    x = rounded(x, DT[dt])
    codes, scales = run_quantize(x, DT[dt], layout, pad)
    want, ws = P.quantize(x)
    assert np.array_equal(codes, P.pack(want))
    assert np.array_equal(scales, P.tile_scales(ws) if layout else ws)


def test_quantize_extremes():
    """The largest and smallest numbers, subnormals, infinities and a NaN beside numbers."""
    big, tiny = np.finfo(np.float32).max, np.float32(1e-45)
    x = np.zeros((1, 6, 64))
    x[0, 0, :32] = big
    x[0, 0, 32:] = tiny
    x[0, 1, :32:2] = -big
    x[0, 1, 32:] = np.float32(2.0 ** -126)
    x[0, 2, 5] = np.float32(2.0 ** -128)
    x[0, 2, 33] = -tiny
    x[0, 3, 0] = np.inf
    x[0, 3, 1] = -np.inf
    x[0, 3, 2] = big
    x[0, 4, :] = np.linspace(-3, 3, 64, dtype=np.float32)
    x[0, 4, 7] = np.nan
    codes, scales = run_quantize(x, torch.float32, 0)
    ok = [0, 1, 2, 5]
    want, ws = P.quantize(x[:, ok])
    assert np.array_equal(scales[:, ok], ws) and np.array_equal(codes[:, ok], P.pack(want))
    got = P.unpack(codes)
    assert got[0, 3, 0] == 7 and got[0, 3, 1] == 15
    rest = np.delete(np.arange(64), 7)
    y = np.where(np.isnan(x), 0.0, x)
    want, ws = P.quantize(y[:, 4:5])
    assert np.array_equal(got[:, 4:5][..., rest], want[..., rest]) and np.array_equal(scales[:, 4:5], ws)


def test_quantize_matches_dispatch():
    """The rows of moe_dispatch in quant_mode 4 with FP4 codes are this quantiser's."""
    W, bs, h, K, E = 2, 9, 256, 2, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(W, bs, h, generator=g, device="cuda").bfloat16()
    ids = torch.rand(W, bs, E, generator=g, device="cuda").topk(K, -1).indices.int().contiguous()
    cfg = M.config(W, bs, h, K, E, torch.bfloat16, quant_mode=4, expand_dtype="fp4_e2m1")
    ws = M.alloc_workspace(cfg)
    out = M.alloc_dispatch_outputs(cfg, torch.bfloat16, expand_scales=False)
    M.dispatch(cfg, x, ids, None, None, out["expand_x"], out["dynamic_scales"], out["assist_info"], out["ep_recv_count"], None, None, ws)
    codes, scales = M.alloc_mx(x)
    M.mx_quantize(x, codes, scales)
    assert M.get_device_status(ws) == 0
    for d in range(W):
        n = int(out["ep_recv_count"][d, -1])
        s, t = out["assist_info"][d, :n, 0].long(), out["assist_info"][d, :n, 1].long()
        assert torch.equal(out["expand_x"][d, :n], codes[s, t])
        assert torch.equal(out["dynamic_scales"][d, :n], scales[s, t])


# ------------------------------------------------------------------ the product

class Product:
    """A random product problem: counts[e] rows for expert e (spread over the source
    ranks), garbage with NaN scales in the rows that no count covers."""

    def __init__(self, W, bs, K_top, counts, n, k, seed, sigma=1.0):
        rng = np.random.default_rng(seed)
        self.W, self.n, self.k, self.E = W, n, k, len(counts)
        L = self.E // W
        self.cfg = M.config(W, bs, max(k, 2), K_top, self.E, torch.bfloat16, quant_mode=4, expand_dtype="fp4_e2m1")
        self.A = M.workspace_size(self.cfg)[1]
        self.ep = np.zeros((W, L * W), dtype=np.int32)
        self.ranges = []
        for d in range(W):
            at = 0
            for le in range(L):
                c = counts[d * L + le]
                cut = np.sort(rng.integers(0, c + 1, W - 1))
                self.ep[d, le * W : le * W + W] = at + np.append(cut, c)
                self.ranges.append((d, at, at + c))
                at += c
            assert at <= self.A
        self.xc = rng.integers(0, 256, (W, self.A, k // 2), dtype=np.uint8)
        self.xs = np.full((W, self.A, k // 32), 255, dtype=np.uint8)
        for d, lo, hi in self.ranges:
            codes, s = P.quantize(rng.standard_normal((hi - lo, k)).astype(np.float32) * sigma)
            self.xc[d, lo:hi], self.xs[d, lo:hi] = P.pack(codes), s
        wc, self.ws = P.quantize(rng.standard_normal((self.E, n, k)).astype(np.float32) / np.sqrt(k))
        self.wc = P.pack(wc)

    def device(self):
        cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return cu(self.xc), cu(self.xs), cu(self.ep), cu(self.wc), cu(P.tile_scales(self.ws))

    def plain(self, e):
        """z and the sums of absolute products of expert e's rows."""
        d, lo, hi = self.ranges[e]
        x = P.values(P.unpack(self.xc[d, lo:hi]), self.xs[d, lo:hi])
        w = P.values(P.unpack(self.wc[e]), self.ws[e])
        return x @ w.T, np.abs(x) @ np.abs(w).T


def run_product(pr, dtype, swiglu, stream=None, expect="OK", ep=None):
    x, xs, ep_dev, w, wsf = pr.device()
    if ep is not None:
        ep_dev = torch.from_numpy(ep).cuda()
    c = pr.n // 2 if swiglu else pr.n
    ws = M.alloc_workspace(pr.cfg)
    ys = None
    if dtype == "fp4":
        y = torch.full((pr.W, pr.A, c // 2), 0xA5, dtype=torch.uint8, device="cuda")
        ys = torch.full((pr.W, pr.A, -(-c // 32)), 0xA5, dtype=torch.uint8, device="cuda")
    else:
        y = torch.full((pr.W, pr.A, c), 777.0, dtype=DT[dtype], device="cuda")
    torch.cuda.synchronize()
    M.expert_product(pr.cfg, x, xs, ep_dev, w, wsf, y, ys, M.EPI_SWIGLU if swiglu else M.EPI_NONE, ws, stream)
    torch.cuda.synchronize()
    assert M.STATUS[M.get_device_status(ws)] == expect
    return y, ys


def product_want(pr, e, swiglu):
    """(result, tolerance) of expert e before the rounding to the output type: fp32 sums of exact
    products, in any order, keep 2^-20 of the sum of magnitudes (16 ulps); SwiGLU has slope at most 1.1
    in the gate, times |up|, and |silu(gate)| in up."""
    z, size = pr.plain(e)
    err = size * 2.0 ** -20
    if not swiglu:
        return z, err
    g, u = z[:, 0::2], z[:, 1::2]
    h = P.silu_gate(z)
    return h, 1.1 * err[:, 0::2] * (np.abs(u) + err[:, 1::2]) + (np.abs(g) + err[:, 0::2]) * err[:, 1::2] + 8 * EPS * np.abs(h)


PRODUCT_CASES = [
    # W, bs, topk, counts, n, k, swiglu
    (2, 4, 2, [1, 0, 0, 0], 64, 32, False),
    (2, 4, 2, [1, 2, 3, 4], 128, 64, False),
    (2, 8, 2, [0, 16, 5, 1], 130, 96, False),
    (2, 8, 2, [3, 0, 0, 16], 1, 160, False),
    (2, 64, 2, [128, 1, 64, 33], 256, 256, False),
    (2, 80, 2, [129, 31, 160, 0], 514, 288, False),
    (2, 150, 2, [300, 0, 257, 7], 320, 512, False),
    (4, 8, 3, [5, 1, 0, 9, 32, 2, 7, 1], 30, 1024, False),
    (2, 4, 2, [1, 0, 0, 0], 64, 32, True),
    (2, 8, 2, [2, 7, 0, 16], 2, 64, True),
    (2, 64, 2, [128, 1, 64, 33], 256, 256, True),
    (2, 80, 2, [129, 31, 0, 160], 516, 320, True),
    (2, 150, 2, [300, 0, 257, 7], 192, 2048, True),
    (4, 16, 3, [5, 1, 0, 9, 32, 2, 7, 1], 1024, 128, True),
    (2, 4, 1, [4, 4], 96, 7168, True),
    (8, 1, 8, [0] * 15 + [1], 1024, 2048, True),
    # several units a CTA, with one, two, three and five stages each (the ring's places shift from unit to unit)
    (2, 75, 2, [150, 5, 140, 129], 8200, 96, False),
    (2, 75, 2, [150, 5, 140, 129], 8192, 512, True),
    (2, 75, 2, [150, 5, 140, 129], 8192, 768, True),
    (2, 75, 2, [150, 5, 140, 129], 4104, 1184, False),
    # every expert with few rows, many units a CTA
    (2, 20, 2, [16, 5, 9, 40], 16384, 768, False),
    (2, 20, 2, [31, 1, 32, 7], 12288, 1280, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("case", PRODUCT_CASES, ids=lambda c: f"w{c[0]}_n{c[4]}_k{c[5]}_{'swiglu' if c[6] else 'plain'}_{max(c[3])}")
def test_product(case, dtype):
    W, bs, topk, counts, n, k, swiglu = case
    if dtype == "fp4" and (n // 2 if swiglu else n) % 2:
        pytest.skip("codes come in pairs")
    pr = Product(W, bs, topk, counts, n, k, seed=n + k)
    y, ys = run_product(pr, dtype, swiglu)
    written = np.zeros((pr.W, pr.A), dtype=bool)
    for e, (d, lo, hi) in enumerate(pr.ranges):
        written[d, lo:hi] = True
        if hi == lo:
            continue
        want, tol = product_want(pr, e, swiglu)
        if dtype == "fp4":
            check_fp4(y[d, lo:hi].cpu().numpy(), ys[d, lo:hi].cpu().numpy(), want, tol)
        else:
            got = y[d, lo:hi].double().cpu().numpy()
            tiny = 2.0 ** -25 if dtype == "f16" else 1e-40
            assert (np.abs(got - want) <= tol + HALF_ULP[dtype] * (np.abs(want) + tol) + tiny).all(), (e, np.abs(got - want).max())
    rest = torch.from_numpy(~written).cuda()
    assert bool((y[rest] == (0xA5 if dtype == "fp4" else 777.0)).all()), "rows beyond the counts were written"
    assert ys is None or bool((ys[rest] == 0xA5).all())


def check_fp4(packed, sbytes, want, tol):
    """Scales and codes of results known to within tol: each scale is that of some amax in range, each value
    within half a step of the number (a step is 0.5, 1 or 2 times X by magnitude; above 6 X it saturates)."""
    c = want.shape[1]
    B = -(-c // 32)
    pad = lambda a: np.pad(a, ((0, 0), (0, B * 32 - c))).reshape(a.shape[0], B, 32)  # noqa: E731
    w, t = pad(want), pad(tol)
    lo, hi = np.abs(w).max(-1) - t.max(-1), np.abs(w).max(-1) + t.max(-1)
    byte = lambda a: np.where(a > 0, np.clip(np.frexp(np.maximum(a, 1e-300))[1] - 3, -127, 127) + 127, 0)  # noqa: E731
    s = sbytes.astype(np.int64)
    assert ((s >= byte(lo)) & (s <= byte(hi))).all()
    X = np.exp2(s - 127.0)[..., None]
    v = pad(P.values(P.unpack(packed), sbytes))
    m = np.abs(w) / X
    step = np.where(m <= 2, 0.5, np.where(m <= 4, 1.0, 2.0))
    near = np.where(m >= 6, m - 6 + 1e-9, step / 2) * X
    # a number within tol of a step's edge may round by the wider step beside it
    assert (np.abs(v - w) <= near * (1 + 1e-6) + 2 * t).all()


def test_product_wide_scales_and_zero_blocks():
    """Scale bytes over a wide range, blocks of zeros with scale byte 0."""
    pr = Product(2, 8, 2, [9, 3, 16, 1], 128, 256, seed=77)
    rng = np.random.default_rng(1)
    for d, lo, hi in pr.ranges:
        pr.xs[d, lo:hi] = rng.integers(97, 158, pr.xs[d, lo:hi].shape)
        pr.xc[d, lo:hi, 16:32] = 0
        pr.xs[d, lo:hi, 1] = 0
    y, _ = run_product(pr, "bf16", False)
    for e, (d, lo, hi) in enumerate(pr.ranges):
        want, tol = product_want(pr, e, False)
        got = y[d, lo:hi].double().cpu().numpy()
        assert (np.abs(got - want) <= tol + HALF_ULP["bf16"] * np.abs(want) + tol).all()


def test_product_same_bytes_on_a_side_stream_and_from_a_graph():
    pr = Product(2, 80, 2, [129, 31, 0, 160], 512, 320, seed=5)
    a, _ = run_product(pr, "bf16", True)
    b, _ = run_product(pr, "bf16", True, stream=torch.cuda.Stream())
    assert torch.equal(a, b)
    x, xs, ep, w, wsf = pr.device()
    y = torch.full_like(a, 777.0)
    ws = M.alloc_workspace(pr.cfg)
    M.expert_product(pr.cfg, x, xs, ep, w, wsf, y, None, M.EPI_SWIGLU, ws)
    torch.cuda.synchronize()
    y.fill_(777.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.expert_product(pr.cfg, x, xs, ep, w, wsf, y, None, M.EPI_SWIGLU, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, y) and M.get_device_status(ws) == 0


@pytest.mark.parametrize("bad", ["above", "negative", "decreasing"])
def test_product_reports_bad_counts(bad):
    pr = Product(2, 8, 2, [3, 4, 5, 6], 64, 64, seed=2)
    ep = pr.ep.copy()
    if bad == "above":
        ep[1, -1] = pr.A + 1
    elif bad == "negative":
        ep[0, 1] = -1
    else:
        ep[0, 3] = ep[0, 1] - 1
    run_product(pr, "bf16", False, expect="BAD_ASSIST", ep=ep)


def test_streams_by_object_and_by_handle():
    rc = M.router_config(300, 64, 4, torch.float32)
    x = torch.randn(300, 64, device="cuda")
    got = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream, 0):
        ids, w = torch.full((300, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(300, 4, device="cuda")
        torch.cuda.synchronize()
        M.route(rc, x, None, ids, w, stream=stream)
        torch.cuda.synchronize()
        got.append((ids, w))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)
    with pytest.raises((TypeError, AttributeError)):
        M.route(rc, x, None, *got[0], stream="side")


def test_product_passes_over_counts_that_overlap_many_times():
    """Counts that fall to zero and rise again at every other expert give some thousand row tiles, of a
    hundred that the units are numbered for."""
    pr = Product(2, 128, 4, [1] * 128, 64, 64, seed=3)
    ep = np.zeros((2, 64, 2), dtype=np.int32)
    ep[:, ::2] = pr.A
    y, _ = run_product(pr, "bf16", False, expect="BAD_ASSIST", ep=ep.reshape(2, 128))
    assert bool((y == 777.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp4"])
def test_product_swiglu_of_large_negative_gates(dtype):
    """silu(-88) is 5e-37: next to an up value of 2^100 and more it still counts. A gate of -inf is out of range
    of the inputs; one of -2^20 gives zero."""
    pr = Product(2, 4, 2, [3, 2, 0, 1], 4, 64, seed=4)
    pr.xc[:], pr.xs[:] = 0, 127
    pr.xc[..., 0] = 0x22  # 1, 1
    gate, up = np.zeros((2, 64)), np.zeros((2, 64))
    gate[0, :2], gate[1, 0] = (-64, -24), -(2.0 ** 20)
    up[0, 0], up[1, 0] = 2.0 ** 120, 2.0 ** 60
    codes, s = P.quantize(np.stack([gate[0], up[0], gate[1], up[1]]))
    pr.wc[:], pr.ws[:] = P.pack(codes), s
    y, ys = run_product(pr, dtype, True)
    want = -88.0 * np.exp(-88.0) / (1 + np.exp(-88.0)) * 2.0 ** 120
    for d, lo, hi in pr.ranges:
        if dtype == "fp4":
            got = P.values(P.unpack(y[d, lo:hi].cpu().numpy()), ys[d, lo:hi].cpu().numpy())
            err = 2.0 ** -3  # half a step of 1 at 4 and above, or of 0.5 at 2 and above
        else:
            got, err = y[d, lo:hi].double().cpu().numpy(), HALF_ULP[dtype]
        # exp's result is below the normal numbers: 2^-149 of 2^-127, and 88 / 2^23 of its value
        assert (np.abs(got[:, 0] - want) <= (err + 2.0 ** -16) * abs(want)).all(), (got[:, 0], want)
        assert (got[:, 1] == 0).all()


def test_product_of_no_tokens():
    cfg = M.config(2, 0, 64, 2, 4, torch.bfloat16, quant_mode=4, expand_dtype="fp4_e2m1")
    ws = M.alloc_workspace(cfg)
    e = torch.empty(2, 0, 32, dtype=torch.uint8, device="cuda")
    w = torch.zeros(4, 8, 32, dtype=torch.uint8, device="cuda")
    M.expert_product(cfg, e, e[..., :2].contiguous(), torch.zeros(2, 4, dtype=torch.int32, device="cuda"), w,
                     torch.zeros(4, 1, 1, 512, dtype=torch.uint8, device="cuda"),
                     torch.empty(2, 0, 8, dtype=torch.bfloat16, device="cuda"), ws=ws)
    assert M.get_device_status(ws) == 0


def test_refusals():
    """What the C entries refuse before launching anything."""
    f = torch.zeros(4, 64, device="cuda")
    ids, w = torch.zeros(4, 8, dtype=torch.int32, device="cuda"), torch.zeros(4, 8, device="cuda")

    def code(call, *a, **k):
        with pytest.raises(M.MoeError) as ei:
            call(*a, **k)
        return ei.value.name

    rc = M.router_config(4, 64, 8, torch.float32)
    M.route(rc, f, None, ids, w)
    for field, value in (("tokens", -1), ("expert_num", 0), ("topk", 0), ("topk", 33), ("group_num", 0), ("group_num", 5),
                         ("topk_group", 0), ("topk_group", 2), ("group_score", 2), ("score_func", 2), ("renormalize", 2),
                         ("logits_dtype", 0), ("scaling", float("inf")), ("logits_stride", 63)):
        bad = M.RouterConfig.from_buffer_copy(rc)
        setattr(bad, field, value)
        L = M.lib()
        assert M.STATUS[L.moe_route(ctypes.byref(bad), f.data_ptr(), None, ids.data_ptr(), w.data_ptr(), None)] == "INVALID_ARG", field
        assert M.STATUS[L.moe_route_backward(ctypes.byref(bad), f.data_ptr(), ids.data_ptr(), w.data_ptr(), f.data_ptr(), 64, None)] == "INVALID_ARG", field
    with pytest.raises(ValueError):
        M.route(rc, f.bfloat16(), None, ids, w)
    with pytest.raises(ValueError):
        M.route(rc, f[:, ::2], None, ids, w)
    with pytest.raises(ValueError):
        M.route(rc, f, None, ids[:, :4], w)

    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    codes, scales = M.alloc_mx(x)
    with pytest.raises(ValueError):
        M.mx_quantize(x, codes, scales[:, :1])
    with pytest.raises(ValueError):
        M.mx_quantize(x.t(), codes, scales)
    assert code(M.mx_quantize, x[:, :63], codes[:, :31].contiguous(), scales) == "INVALID_ARG"  # an odd number of columns

    pr = Product(2, 8, 2, [3, 4, 5, 6], 64, 64, seed=2)
    x, xs, ep, wt, wsf = pr.device()
    ws = M.alloc_workspace(pr.cfg)
    y = torch.empty(2, pr.A, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        M.expert_product(pr.cfg, x, xs, ep, wt, wsf[:2], y, ws=ws)
    with pytest.raises(ValueError):
        M.expert_product(pr.cfg, x, xs, ep, wt, wsf, y[..., :32].contiguous(), ws=ws)
    assert code(M.expert_product, pr.cfg, x, xs, ep, wt, wsf, y.int(), ws=ws) == "INVALID_ARG"
    assert code(M.expert_product, pr.cfg, x, xs, ep, wt, wsf, y, epilogue=2, ws=ws) == "INVALID_ARG"
    assert code(M.expert_product, pr.cfg, x, xs, ep, wt, wsf, y, ws=ws[:-256]) == "WORKSPACE"
    y4 = torch.empty(2, pr.A, 32, dtype=torch.uint8, device="cuda")
    assert code(M.expert_product, pr.cfg, x, xs, ep, wt, wsf, y4, ws=ws) == "INVALID_ARG"  # no scales for the codes
    w48 = torch.zeros(4, 64, 24, dtype=torch.uint8, device="cuda")
    x48 = torch.zeros(2, pr.A, 24, dtype=torch.uint8, device="cuda")
    assert code(M.expert_product, pr.cfg, x48, xs[..., :1].contiguous(), ep, w48, wsf, y, ws=ws) == "UNSUPPORTED"  # k = 48
