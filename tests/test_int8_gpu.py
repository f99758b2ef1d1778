"""int8 rows (include/moe_experts.h): the quantiser's bytes against IEEE arithmetic in
numpy, the experts' product against integer sums and 64-bit scales."""
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
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def code(call, *a, **k):
    with pytest.raises(M.MoeError) as ei:
        call(*a, **k)
    return ei.value.name


# ------------------------------------------------------------------ quantisation

def quantized(x):
    """Codes and scales of a float32 array by numpy's IEEE divisions."""
    amax = np.nanmax(np.abs(x), axis=-1, initial=0.0).astype(np.float32)
    scale = (amax / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        q = np.rint((x / scale[..., None]).astype(np.float32))
    q = np.where(np.isnan(q), 0, q)
    return np.clip(q, -127, 127).astype(np.int8), scale


def make_rows(rng, shape, dtype, std=1.0):
    x = torch.from_numpy(rng.standard_normal(shape) * std).to(DT[dtype])
    return x, x.float().numpy()


QUANT_SHAPES = [(1, 1, 1), (3, 5, 7), (2, 3, 8), (1, 9, 250), (2, 33, 256), (2, 10, 264), (1, 40, 512), (3, 7, 1000), (2, 17, 1024),
                (1, 19, 2048), (1, 5, 2056), (2, 3, 4090), (1, 4, 7168), (1, 3, 8192), (1, 3, 9000), (1, 2, 16384), (1, 2, 20001),
                (700, 2, 16), (1, 5000, 24),
                (2, 300, 511), (1, 90, 2046), (1, 90, 2047), (1, 20, 8190), (1, 9, 16383), (3, 5, 18432), (1, 700, 18430),
                (1, 700, 16385), (2, 9, 32768), (1, 5, 32766), (1, 3, 32769), (2, 90, 40000), (1, 30, 40002), (1, 9, 65535)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", QUANT_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_quantize(shape, dtype):
    rng = np.random.default_rng(sum(shape))
    x, xf = make_rows(rng, shape, dtype)
    codes, scales = M.alloc_int8(x.cuda())
    M.int8_quantize(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    q, s = quantized(xf)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (24, 8), (3, 5)])
@pytest.mark.parametrize("cols", [64, 100, 2048])
def test_quantize_strided_rows(cols, pad, offset, dtype):
    rng = np.random.default_rng(cols + pad)
    mats, rows = 3, 6
    whole = torch.full((mats * (rows + 1) * (cols + pad) + offset,), float("inf"), dtype=DT[dtype], device="cuda")
    x = whole[offset:].view(mats, rows + 1, cols + pad)[:, :rows, :cols]
    host, xf = make_rows(rng, (mats, rows, cols), dtype)
    x.copy_(host)
    codes, scales = M.alloc_int8(x)
    M.int8_quantize(x, codes, scales)
    torch.cuda.synchronize()
    q, s = quantized(xf)
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), q)


@pytest.mark.parametrize("cols", [40, 41, 4096])
def test_quantize_edges(cols):
    """Zeros, infinities, NaN, values at half steps, rows whose scale is subnormal."""
    x = np.zeros((8, cols), dtype=np.float32)
    rng = np.random.default_rng(cols)
    x[1] = rng.standard_normal(cols)
    x[1, 3] = np.inf
    x[2] = rng.standard_normal(cols)
    x[2, 5] = np.nan
    x[3] = np.nan
    x[4] = np.arange(cols) % 254 - 126.5  # amax 127 at most by the next line: a scale of 1, all ties
    x[4, 0] = 127.0
    x[5] = rng.standard_normal(cols) * 1e-42
    x[6] = rng.standard_normal(cols) * 1e-37
    x[7] = rng.standard_normal(cols) * 3e37
    t = torch.from_numpy(x).cuda()
    codes, scales = M.alloc_int8(t)
    M.int8_quantize(t, codes, scales)
    torch.cuda.synchronize()
    q, s = quantized(x)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(scales, s)
    there = ~np.isnan(x)
    assert np.array_equal(codes[there], q[there])
    assert scales[1] == np.inf and not codes[1].any() and scales[3] == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_edges_of_16_bits(dtype):
    """The largest magnitude is taken pair by pair there: NaN in either half, infinities, the type's ends, zeros."""
    cols, t = 64, DT[dtype]
    x = torch.randn(9, cols, generator=torch.Generator().manual_seed(3)).to(t)
    x[0], x[1, 7], x[2, 8], x[3] = 0, float("nan"), float("nan"), float("nan")
    x[4, 63], x[5, 62] = float("inf"), -float("inf")
    x[6, 5], x[7] = torch.finfo(t).min, torch.finfo(t).tiny / 4 if dtype == "f16" else 1e-40
    x[8, 11] = 0.0
    codes, scales = M.alloc_int8(x.cuda())
    M.int8_quantize(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    q, s = quantized(x.float().numpy())
    there = ~torch.isnan(x).numpy()
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy()[there], q[there])


@pytest.mark.parametrize("cols", [256, 250])
@pytest.mark.parametrize("exponent", [-140, -126, -101, -100, -90, -3, 0, 40, 119])
def test_quantize_next_to_half_steps(exponent, cols):
    """Elements whose quotient is half a step and its neighbours in fp32, at scales from the smallest to the largest."""
    rng = np.random.default_rng(exponent + 200)
    rows = 400
    scale = np.ldexp(rng.uniform(1, 2, rows), exponent).astype(np.float32)
    x = np.zeros((rows, cols), dtype=np.float32)
    amax = (scale * np.float32(127)).astype(np.float32)
    x[:, 0] = np.where(np.isfinite(amax), amax, np.float32(3.4e38))
    scale = (x[:, 0] / np.float32(127)).astype(np.float32)
    half = rng.integers(-127, 127, (rows, cols - 1)) + 0.5
    near = (half * scale[:, None].astype(np.float64)).astype(np.float32)
    for _ in range(2):  # up to two steps of fp32 to either side
        step = rng.integers(-1, 2, near.shape)
        near = np.where(step < 0, np.nextafter(near, np.float32(-np.inf)), np.where(step > 0, np.nextafter(near, np.float32(np.inf)), near))
    x[:, 1:] = np.clip(near, -x[:, :1], x[:, :1])
    t = torch.from_numpy(x).cuda()
    codes, scales = M.alloc_int8(t)
    M.int8_quantize(t, codes, scales)
    torch.cuda.synchronize()
    q, s = quantized(x)
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), q)


@pytest.mark.parametrize("cols,dtype", [(64, "bf16"), (66, "f16"), (4096, "f32"), (3000, "bf16")])
def test_quantize_received_rows(cols, dtype):
    """With counts, rows beyond the last count of a rank are neither read nor written."""
    rng = np.random.default_rng(cols)
    last = [0, 5, 13, -4, 99, 1]
    W, A = len(last), 13
    ep = torch.randint(0, 5, (W, 4), dtype=torch.int32)
    ep[:, -1] = torch.tensor(last)
    host, xf = make_rows(rng, (W, A, cols), dtype)
    x = host.cuda()
    codes, scales = torch.full((W, A, cols), 99, dtype=torch.int8, device="cuda"), torch.full((W, A), -7.0, device="cuda")
    M.int8_quantize(x, codes, scales, ep_recv_count=ep.cuda())
    torch.cuda.synchronize()
    q, s = quantized(xf)
    for d, n in enumerate(last):
        n = min(max(n, 0), A)
        assert np.array_equal(codes[d, :n].cpu().numpy(), q[d, :n]) and np.array_equal(scales[d, :n].cpu().numpy(), s[d, :n])
        assert bool((codes[d, n:] == 99).all()) and bool((scales[d, n:] == -7.0).all())


def test_quantize_as_dispatch_does():
    cfg = M.config(2, 40, 264, 2, 4, torch.bfloat16, quant_mode=2)
    ws, out = M.alloc_workspace(cfg), M.alloc_dispatch_outputs(cfg, torch.bfloat16)
    x = torch.randn(2, 40, 264, device="cuda").bfloat16()
    ids = torch.stack([torch.randperm(4, device="cuda")[:2] for _ in range(80)]).int().view(2, 40, 2)
    w = torch.rand(2, 40, 2, device="cuda")
    M.dispatch(cfg, x, ids, None, w, out["expand_x"], out["dynamic_scales"], out["assist_info"], out["ep_recv_count"],
               out["expand_scales"], None, ws)
    codes, scales = M.alloc_int8(x)
    M.int8_quantize(x, codes, scales)
    assert M.get_device_status(ws) == 0
    for d in range(2):
        n = int(out["ep_recv_count"][d, -1])
        s, t, _ = out["assist_info"][d, :n].long().unbind(-1)
        assert torch.equal(out["expand_x"][d, :n], codes[s, t]) and torch.equal(out["dynamic_scales"][d, :n], scales[s, t])


# ------------------------------------------------------------------ the product

class Product:
    """Rows and weights with given row counts an expert (W ranks, experts in turn)."""

    def __init__(self, W, bs, topk, counts, n, k, seed=0):
        rng = np.random.default_rng(seed)
        E = len(counts)
        L = E // W
        self.W, self.E, self.n, self.k = W, E, n, k
        self.cfg = M.config(W, bs, 64, topk, E, torch.bfloat16, quant_mode=2)
        _, self.A = M.workspace_size(self.cfg)
        self.ep = np.zeros((W, L * W), dtype=np.int32)
        self.ranges = []
        for d in range(W):
            row = 0
            for le in range(L):
                c = counts[d * L + le]
                parts = np.bincount(rng.integers(0, W, c), minlength=W)
                self.ep[d, le * W:(le + 1) * W] = row + np.cumsum(parts)
                self.ranges.append((d, row, row + c))
                row += c
            assert row <= self.A, (row, self.A)
        self.x = rng.integers(-127, 128, (W, self.A, k)).astype(np.int8)
        self.xs = rng.uniform(0.5, 2.0, (W, self.A)).astype(np.float32)
        self.w = rng.integers(-128, 128, (E, n, k)).astype(np.int8)
        self.ws = (rng.uniform(0.5, 2.0, (E, n)) / (5400 * k ** 0.5)).astype(np.float32)

    def run(self, dtype, swiglu, scaled=True, stream=None, expect="OK", ep=None):
        c = self.n // 2 if swiglu else self.n
        y = torch.full((self.W, self.A, c), 777.0, dtype=DT[dtype], device="cuda")
        dev = [torch.from_numpy(a).cuda() for a in (self.x, self.xs, self.ep if ep is None else ep, self.w, self.ws)]
        ws = M.alloc_workspace(self.cfg)
        torch.cuda.synchronize()
        M.expert_product_int8(self.cfg, dev[0], dev[1] if scaled else None, dev[2], dev[3], dev[4], y,
                              M.EPI_SWIGLU if swiglu else M.EPI_NONE, ws, stream)
        torch.cuda.synchronize()
        assert M.STATUS[M.get_device_status(ws)] == expect
        return y

    def want(self, e, swiglu, scaled=True):
        """(result, tolerance) of expert e before the rounding to the output type."""
        d, lo, hi = self.ranges[e]
        x, w = self.x[d, lo:hi].astype(np.float64), self.w[e].astype(np.float64)
        scale = self.ws[e].astype(np.float64) * (self.xs[d, lo:hi, None].astype(np.float64) if scaled else 1.0)
        z = x @ w.T * scale  # whole numbers below 2^53: exact
        # partial sums beyond 2^24 are rounded as they grow, by 2^-24 of the sum of magnitudes for each 16 products at
        # most; two products with the scales
        sums = np.abs(x) @ np.abs(w).T
        err = np.where(sums > 2.0 ** 24, EPS * (self.k / 16 + 1) * sums * scale, 0.0) + 3 * EPS * np.abs(z)
        if not swiglu:
            return z, err
        g, u, eg, eu = z[:, 0::2], z[:, 1::2], err[:, 0::2], err[:, 1::2]
        h = P.silu_gate(z)
        # silu's slope is at most 1.1; the exponential and the reciprocal: within 2^-16 of their size
        return h, 1.1 * eg * (np.abs(u) + eu) + (np.abs(g) + eg) * eu + 2.0 ** -16 * np.abs(h)

    def check(self, y, dtype, swiglu, scaled=True):
        written = np.zeros((self.W, self.A), dtype=bool)
        for e, (d, lo, hi) in enumerate(self.ranges):
            written[d, lo:hi] = True
            if hi == lo:
                continue
            want, tol = self.want(e, swiglu, scaled)
            got = y[d, lo:hi].double().cpu().numpy()
            tiny = 2.0 ** -25 if dtype == "f16" else 1e-40
            off = np.abs(got - want) - (tol + HALF_ULP[dtype] * (np.abs(want) + tol) + tiny)
            assert (off <= 0).all(), (e, np.unravel_index(off.argmax(), off.shape), off.max())
        assert bool((y[torch.from_numpy(~written).cuda()] == 777.0).all()), "rows beyond the counts were written"


PRODUCT_CASES = [
    # W, bs, topk, counts, n, k, swiglu
    (2, 4, 2, [1, 0, 0, 0], 64, 16, False),
    (2, 4, 2, [1, 2, 3, 4], 128, 64, False),
    (2, 8, 2, [0, 16, 5, 1], 130, 96, False),
    (2, 8, 2, [3, 0, 0, 16], 1, 160, False),
    (2, 8, 2, [3, 0, 0, 16], 33, 7, False),
    (2, 24, 2, [33, 5, 0, 48], 70, 129, True),
    (2, 64, 2, [128, 1, 64, 33], 256, 256, False),
    (2, 80, 2, [129, 31, 160, 0], 514, 272, False),
    (2, 150, 2, [300, 0, 257, 7], 320, 512, False),
    (4, 8, 3, [5, 1, 0, 9, 32, 2, 7, 1], 30, 1024, False),
    (2, 4, 2, [1, 0, 0, 0], 64, 32, True),
    (2, 8, 2, [2, 7, 0, 16], 2, 64, True),
    (2, 64, 2, [128, 1, 64, 33], 256, 256, True),
    (2, 80, 2, [129, 31, 0, 160], 516, 336, True),
    (2, 150, 2, [300, 0, 257, 7], 192, 2048, True),
    (4, 16, 3, [5, 1, 0, 9, 32, 2, 7, 1], 1024, 128, True),
    (2, 4, 1, [4, 4], 96, 7168, True),
    (8, 1, 8, [0] * 15 + [1], 1024, 2048, True),
    # several units a CTA, of few and many stages
    (2, 75, 2, [150, 5, 140, 129], 8200, 96, False),
    (2, 75, 2, [150, 5, 140, 129], 8192, 512, True),
    (2, 75, 2, [150, 5, 140, 129], 4104, 1200, False),
    (2, 300, 2, [600, 0, 513, 31], 2050, 400, False),
    (2, 300, 2, [600, 17, 513, 0], 2080, 640, True),
    # every expert with few rows, many units a CTA
    (2, 20, 2, [16, 5, 9, 40], 16384, 768, False),
    (2, 20, 2, [31, 1, 32, 7], 12288, 1280, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", PRODUCT_CASES, ids=lambda c: f"w{c[0]}_n{c[4]}_k{c[5]}_{'swiglu' if c[6] else 'plain'}_{max(c[3])}")
def test_product(case, dtype):
    W, bs, topk, counts, n, k, swiglu = case
    pr = Product(W, bs, topk, counts, n, k, seed=n + k)
    pr.check(pr.run(dtype, swiglu), dtype, swiglu)


@pytest.mark.parametrize("case", [
    (2, 4, 1, [0, 8], 33, 129, False), (2, 4, 1, [8, 0], 1, 1, False), (2, 4, 1, [3, 8], 65, 131, False), (2, 4, 1, [1, 8], 63, 127, False),
    (2, 40, 1, [5, 80], 65, 2047, False), (2, 40, 1, [80, 33], 130, 1001, True), (2, 4, 1, [8, 8], 2, 257, True),
    (2, 16, 1, [32, 1], 129, 2040, False), (2, 16, 1, [31, 32], 66, 4095, True), (2, 100, 1, [200, 7], 1023, 385, False),
], ids=lambda c: f"n{c[4]}_k{c[5]}_{'swiglu' if c[6] else 'plain'}")
def test_product_of_odd_lengths(case):
    """Rows that begin at every byte of a word, matrices that end inside one, a full rank's last row."""
    W, bs, topk, counts, n, k, swiglu = case
    pr = Product(W, bs, topk, counts, n, k, seed=n + k)
    for dtype in ("bf16", "f16"):
        pr.check(pr.run(dtype, swiglu), dtype, swiglu)


@pytest.mark.parametrize("k", [1024, 1000, 336])
def test_product_sums_are_whole(k):
    """Sums that grow to millions and come back to a few units: exact up to k = 1024."""
    pr = Product(2, 40, 2, [40, 3, 0, 77], 256, k, seed=k)
    rng = np.random.default_rng(k)
    half = k // 2
    pr.x[..., half:2 * half] = -pr.x[..., :half]
    pr.x[:, ::3, :half], pr.x[:, ::3, half:2 * half] = 127, -127
    pr.w[pr.w == -128] = -127
    pr.w[:, ::2, :half] = 127
    pr.w[..., half:2 * half] = pr.w[..., :half]
    at = rng.integers(0, half, (pr.E, pr.n, 3))
    for e in range(pr.E):
        for j in range(pr.n):
            pr.w[e, j, at[e, j]] -= 1
    pr.xs[:], pr.ws[:] = 1.0, 1.0
    y = pr.run("f16", False)
    for e, (d, lo, hi) in enumerate(pr.ranges):
        want = pr.x[d, lo:hi].astype(np.int64) @ pr.w[e].astype(np.int64).T
        assert np.abs(want).max(initial=0) < 2048  # f16 holds them
        assert np.array_equal(y[d, lo:hi].cpu().numpy().astype(np.int64), want)


@pytest.mark.parametrize("k", [4096, 131071, 131056])
def test_product_largest_sums(k):
    """All codes at the ends of their range, over the longest rows."""
    pr = Product(2, 2, 1, [2, 1], 6, k, seed=1)
    pr.x[:], pr.w[:] = -128, -128
    pr.w[:, 1::2] = 127
    pr.xs[:], pr.ws[:] = 2.0 ** -13, 2.0 ** -13
    y = pr.run("bf16", False)
    for e, (d, lo, hi) in enumerate(pr.ranges):
        want = pr.x[d, lo:hi].astype(np.float64) @ pr.w[e].astype(np.float64).T * 2.0 ** -26
        got = y[d, lo:hi].double().cpu().numpy()
        # an addition of 16 products may be cut instead of rounded: one step of fp32 each
        assert (np.abs(got - want) <= (2.0 ** -8 + 2 * EPS * (k / 16 + 1)) * np.abs(want)).all()


@pytest.mark.parametrize("k", [64, 67])
def test_product_of_no_rows(k):
    """Tokens that all went elsewhere: counts of zero, and one expert with a row among many without."""
    for counts in ([0, 0, 0, 0], [0, 0, 1, 0]):
        pr = Product(2, 8, 2, counts, 96, k, seed=8)
        pr.check(pr.run("bf16", False), "bf16", False)


def test_product_calls_that_overlap():
    """Two streams, one workspace: the product writes nothing there."""
    a, b = Product(2, 80, 2, [129, 31, 0, 160], 512, 320, seed=5), Product(2, 80, 2, [3, 90, 100, 1], 512, 320, seed=6)
    want = [pr.run("bf16", True) for pr in (a, b)]
    dev = [[torch.from_numpy(t).cuda() for t in (pr.x, pr.xs, pr.ep, pr.w, pr.ws)] for pr in (a, b)]
    ys, ws = [torch.full_like(w, 777.0) for w in want], M.alloc_workspace(a.cfg)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, y, st in zip(dev, ys, streams):
            M.expert_product_int8(a.cfg, *d, y, M.EPI_SWIGLU, ws, st)
    torch.cuda.synchronize()
    assert M.get_device_status(ws) == 0 and all(torch.equal(y, w) for y, w in zip(ys, want))


def test_product_without_row_scales():
    pr = Product(2, 80, 2, [129, 31, 0, 160], 130, 320, seed=5)
    pr.check(pr.run("bf16", False, scaled=False), "bf16", False, scaled=False)


def test_product_infinite_and_nan_scales_stay_in_their_row_and_channel():
    pr = Product(2, 40, 2, [40, 3, 0, 77], 64, 64, seed=6)
    pr.xs[0, 1], pr.ws[0, 5] = np.inf, np.nan
    y = pr.run("f16", False).float().cpu().numpy()
    clean = np.isfinite(y[0, :40])
    assert not clean[1].any() and not clean[:, 5].any()
    clean[1], clean[:, 5] = True, True
    assert clean.all() and np.isfinite(y[1, :77]).all()


@pytest.mark.parametrize("k", [320, 321])
def test_product_same_bytes_on_a_side_stream_and_from_a_graph(k):
    pr = Product(2, 80, 2, [129, 31, 0, 160], 512, k, seed=5)
    a = pr.run("bf16", True)
    assert torch.equal(a, pr.run("bf16", True, stream=torch.cuda.Stream()))
    dev = [torch.from_numpy(t).cuda() for t in (pr.x, pr.xs, pr.ep, pr.w, pr.ws)]
    y, ws = torch.full_like(a, 777.0), M.alloc_workspace(pr.cfg)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        M.expert_product_int8(pr.cfg, *dev, y, M.EPI_SWIGLU, ws)
    for _ in range(2):
        y.fill_(777.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, y) and M.get_device_status(ws) == 0


@pytest.mark.parametrize("k", [64, 65])
@pytest.mark.parametrize("bad", ["above", "negative", "decreasing"])
def test_product_reports_bad_counts(bad, k):
    pr = Product(2, 8, 2, [3, 4, 5, 6], 64, k, seed=2)
    ep = pr.ep.copy()
    if bad == "above":
        ep[1, -1] = pr.A + 1
    elif bad == "negative":
        ep[0, 1] = -1
    else:
        ep[0, 3] = ep[0, 1] - 1
    pr.run("bf16", False, expect="BAD_ASSIST", ep=ep)


@pytest.mark.parametrize("k", [64, 65])
def test_product_passes_over_counts_that_overlap_many_times(k):
    pr = Product(2, 128, 4, [1] * 128, 64, k, seed=3)
    ep = np.zeros((2, 64, 2), dtype=np.int32)
    ep[:, ::2] = pr.A
    y = pr.run("bf16", False, expect="BAD_ASSIST", ep=ep.reshape(2, 128))
    assert bool((y == 777.0).all())


def test_product_of_no_tokens_and_of_many_experts():
    cfg = M.config(2, 0, 64, 2, 4, torch.bfloat16, quant_mode=2)
    e8 = torch.empty(2, 0, 64, dtype=torch.int8, device="cuda")
    ws = M.alloc_workspace(cfg)
    M.expert_product_int8(cfg, e8, torch.empty(2, 0, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
                          torch.zeros(4, 8, 64, dtype=torch.int8, device="cuda"), torch.ones(4, 8, device="cuda"),
                          torch.empty(2, 0, 8, dtype=torch.bfloat16, device="cuda"), ws=ws)
    assert M.get_device_status(ws) == 0
    rng = np.random.default_rng(9)
    for E in (1000, 1024):
        counts = rng.integers(0, 3, E)
        pr = Product(2, 256, 32, list(counts), 40, 48, seed=9)
        pr.check(pr.run("f16", False), "f16", False)


def test_refusals():
    pr = Product(2, 8, 2, [3, 4, 5, 6], 64, 64, seed=2)
    x, xs, ep, w, wsc = [torch.from_numpy(t).cuda() for t in (pr.x, pr.xs, pr.ep, pr.w, pr.ws)]
    ws = M.alloc_workspace(pr.cfg)
    y = torch.empty(2, pr.A, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((x.int(), xs, ep, w, wsc, y), (x[:, :, :32].contiguous(), xs, ep, w, wsc, y), (x, xs[:1], ep, w, wsc, y),
                 (x, xs.half(), ep, w, wsc, y), (x, xs, ep[:1], w, wsc, y), (x, xs, ep, w, wsc[:2], y),
                 (x, xs, ep, w, wsc, y[..., :32].contiguous()), (x, xs, ep, w, None, y[..., ::2]), (x.cpu(), xs, ep, w, wsc, y)):
        with pytest.raises(ValueError):
            M.expert_product_int8(pr.cfg, *args, ws=ws)
    assert code(M.expert_product_int8, pr.cfg, x, xs, ep, w, wsc, y.float(), ws=ws) == "INVALID_ARG"
    assert code(M.expert_product_int8, pr.cfg, x, xs, ep, w, wsc, y, epilogue=2, ws=ws) == "INVALID_ARG"
    assert code(M.expert_product_int8, pr.cfg, x, xs, ep, w, None, y, ws=ws) == "INVALID_ARG"
    assert code(M.expert_product_int8, pr.cfg, x, xs, ep, w, wsc, y, ws=ws[:-256]) == "WORKSPACE"

    v = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    codes, scales = M.alloc_int8(v)
    for args in ((v.int(), codes, scales), (v, codes[..., :32], scales), (v, codes, scales[:1]), (v.transpose(1, 2), codes, scales),
                 (v[0, 0], codes, scales)):
        with pytest.raises(ValueError):
            M.int8_quantize(*args)
    with pytest.raises(ValueError):
        M.int8_quantize(v, codes, scales, ep_recv_count=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        M.int8_quantize(v, codes, scales, ep_recv_count=torch.zeros(4, device="cuda"))
