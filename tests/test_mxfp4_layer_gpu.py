"""The MX FP4 layer (mxfp4_layer.py): routing, dispatch, the two products and the
combine run together, against the plain 64-bit forms of each step."""
import numpy as np
import pytest
import torch

import experts_plain as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    from combine_route_scan_gb300.mxfp4_layer import Mxfp4Layer
    B.build()


def make(W=4, bs=12, h=256, E=8, K=2, I=64, seed=1, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    wg, wu, wd = (draw(E, I, h) * 0.1).bfloat16(), (draw(E, I, h) * 0.1).bfloat16(), (draw(E, h, I) * 0.1).bfloat16()
    layer = Mxfp4Layer(W, bs, K, wg, wu, wd, **kw)
    return layer, draw(W, bs, h).bfloat16(), draw(W * bs, E), (wg, wu, wd)


def mx(t):
    codes, s = P.quantize(t.double().cpu().numpy())
    return P.values(codes, s)


def test_layer_against_the_plain_steps():
    layer, x, logits, (wg, wu, wd) = make()
    out = layer(x, logits)
    assert M.get_device_status(layer.ws) == 0
    W, bs, h = x.shape
    E, I = wg.shape[:2]
    K = layer.ids.shape[-1]
    L = E // W
    xv, gv, uv, dv = mx(x), mx(wg), mx(wu), mx(wd)
    assist, ep = layer.rows["assist_info"].cpu().numpy(), layer.rows["ep_recv_count"].cpu().numpy()
    ids, weights = layer.ids.cpu().numpy(), layer.weights.double().cpu().numpy()
    lg = logits.double().cpu().numpy()
    for t in range(W * bs):
        ri, rw = P.route_token(lg[t], None, K, 1, 1, False, False, True, 1.0)
        assert np.array_equal(ids.reshape(-1, K)[t], ri)
        assert np.allclose(weights.reshape(-1, K)[t], rw, rtol=2.0 ** -18)
    h1 = P.values(P.unpack(layer.h1.cpu().numpy()), layer.h1_scales.cpu().numpy())
    y = layer.y.double().cpu().numpy()
    want = np.zeros((W, bs, h))
    seen = np.zeros((W, bs, K), dtype=int)
    for d in range(W):
        for r in range(ep[d, -1]):
            le = int(np.searchsorted(ep[d], r, side="right")) // W
            e = d * L + le
            s, t, k = assist[d, r]
            assert ids[s, t, k] == e
            seen[s, t, k] += 1
            g, u = gv[e] @ xv[s, t], uv[e] @ xv[s, t]
            act = g / (1 + np.exp(-g)) * u
            # within half a step of the format at the block's own scale (its largest number is 4 .. 8 X, a step 2 X at most)
            X = np.exp2(layer.h1_scales[d, r].double().cpu().numpy() - 127).repeat(32)[:I]
            assert (np.abs(h1[d, r] - act) <= X * 2 * (1 + 1e-5) + 1e-5).all()
            z = dv[e] @ h1[d, r]
            # sums of 64 exact products in fp32, then one rounding to bf16
            assert (np.abs(y[d, r] - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -18 * (np.abs(dv[e]) @ np.abs(h1[d, r]))).all()
            want[s, t] += weights[s, t, k] * y[d, r]
    assert (seen == 1).all()
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1e-5 * np.abs(want).max()).all()


def test_layer_near_the_bf16_layer():
    """The 4-bit rounding leaves the output within a third of bf16's: a rounding is off by some 0.12 of its number,
    so gate and up are by 0.17 (rows and weights), their product by 0.24, and with its own rounding and w_down's the
    output by 0.30."""
    layer, x, logits, (wg, wu, wd) = make(W=2, bs=32, h=512, E=8, K=2, I=256, router=dict(score_func=M.SCORE_SIGMOID))
    out = layer(x, logits)
    cfg = M.config(2, 32, 512, 2, 8, torch.bfloat16, ffn_intermediate=256)
    ws = M.alloc_workspace(cfg)
    want = torch.empty_like(x)
    M.dispatch_ffn_combine(cfg, x, layer.ids, None, layer.weights, wg, wu, wd, want, ws)
    assert M.get_device_status(ws) == 0 and M.get_device_status(layer.ws) == 0
    assert float((out.float() - want.float()).norm() / want.float().norm()) < 1 / 3


def test_layer_replays_from_a_cuda_graph():
    layer, x, logits, _ = make(seed=3)
    want = layer(x, logits)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and M.get_device_status(layer.ws) == 0


def test_logits_gradient_of_a_step():
    layer, x, logits, _ = make(seed=4, router=dict(renormalize=False))
    layer(x, logits)
    grad = torch.randn(layer.weights.shape, device="cuda")
    got = layer.logits_gradient(logits, grad).double().cpu().numpy()
    ids, lg, g = layer.ids.cpu().numpy().reshape(-1, 2), logits.double().cpu().numpy(), grad.cpu().numpy().reshape(-1, 2)
    for t in range(len(ids)):
        want = P.route_gradient(lg[t], ids[t], g[t], False, False, 1.0)
        assert np.allclose(got[t], want, rtol=0, atol=2.0 ** -18 * np.abs(g[t]).max())


def test_layer_with_groups_and_a_bias():
    """The router's groups and balancing bias reach the layer's choice, its weights the output."""
    from test_experts_gpu import separated_logits
    rng = np.random.default_rng(12)
    W, bs, h, E, K, I = 4, 12, 256, 16, 3, 64
    bias = np.round(rng.uniform(-0.1, 0.1, E), 3).astype(np.float32)
    router = dict(score_func=M.SCORE_SIGMOID, group_num=4, topk_group=2, group_score=M.GROUP_TOP2_SUM, scaling=2.5)
    layer, x, _, (wg, wu, wd) = make(W, bs, h, E, K, I, seed=12, bias=torch.from_numpy(bias).cuda(), router=router)
    lg = separated_logits(rng, W * bs, E, torch.float32, bias, True, K, 4, 2, True)
    out = layer(x, torch.from_numpy(lg).float().cuda())
    assert M.get_device_status(layer.ws) == 0
    ids, weights = layer.ids.cpu().numpy().reshape(-1, K), layer.weights.double().cpu().numpy().reshape(-1, K)
    for t in range(W * bs):
        ri, rw = P.route_token(lg[t], bias, K, 4, 2, True, True, True, 2.5)
        assert np.array_equal(ids[t], ri)
        assert np.allclose(weights[t], rw, rtol=2.0 ** -18)
    cfg = M.config(W, bs, h, K, E, torch.bfloat16, ffn_intermediate=128)
    # the bf16 layer wants 128 features: the others' weights are zeros
    pad = lambda w: torch.nn.functional.pad(w, (0, 0, 0, 128 - I))  # noqa: E731
    ws = M.alloc_workspace(cfg)
    want = torch.empty_like(x)
    M.dispatch_ffn_combine(cfg, x, layer.ids, None, layer.weights, pad(wg).contiguous(), pad(wu).contiguous(),
                           torch.nn.functional.pad(wd, (0, 128 - I)).contiguous(), want, ws)
    assert M.get_device_status(ws) == 0
    # as in test_layer_near_the_bf16_layer
    assert float((out.float() - want.float()).norm() / want.float().norm()) < 1 / 3
