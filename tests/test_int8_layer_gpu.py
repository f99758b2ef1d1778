"""The int8 layer (int8_layer.py): routing, dispatch, the two products and the combine run
together, against the plain 64-bit forms of each step, with the gradient of its router."""
import numpy as np
import pytest
import torch

import experts_plain as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    from combine_route_scan_gb300.int8_layer import Int8Layer
    from combine_route_scan_gb300.mxfp4_layer import Mxfp4Layer
    B.build()

EPS = 2.0 ** -24


def make(W=4, bs=12, h=256, E=8, K=2, I=64, seed=1, kind=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    wg, wu, wd = (draw(E, I, h) * 0.1).bfloat16(), (draw(E, I, h) * 0.1).bfloat16(), (draw(E, h, I) * 0.1).bfloat16()
    layer = (kind or Int8Layer)(W, bs, K, wg, wu, wd, **kw)
    return layer, draw(W, bs, h).bfloat16(), draw(W * bs, E), (wg, wu, wd)


def int8(t):
    """Codes and scales in 64 bits of a bf16 tensor's rows, with fp32's divisions."""
    x = t.float().cpu().numpy()
    scale = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    return np.clip(np.rint((x / scale[..., None]).astype(np.float32)), -127, 127).astype(np.float64), scale.astype(np.float64)


@pytest.mark.parametrize("h,I", [(256, 64), (120, 72), (128, 40)])
def test_layer_against_the_plain_steps(h, I):
    layer, x, logits, (wg, wu, wd) = make(h=h, I=I)
    out = layer(x, logits)
    assert M.get_device_status(layer.ws) == 0
    W, bs, _ = x.shape
    E, K = wg.shape[0], layer.ids.shape[-1]
    L = E // W
    (xq, xs), (gq, gs), (uq, us), (dq, ds) = int8(x), int8(wg), int8(wu), int8(wd)
    assist, ep = layer.rows["assist_info"].cpu().numpy(), layer.rows["ep_recv_count"].cpu().numpy()
    ids, weights = layer.ids.cpu().numpy(), layer.weights.double().cpu().numpy()
    lg = logits.double().cpu().numpy()
    for t in range(W * bs):
        ri, rw = P.route_token(lg[t], None, K, 1, 1, False, False, True, 1.0)
        assert np.array_equal(ids.reshape(-1, K)[t], ri)
        assert np.allclose(weights.reshape(-1, K)[t], rw, rtol=2.0 ** -18)
    h1, y = layer.h1.double().cpu().numpy(), layer.y.double().cpu().numpy()
    codes, scales = layer.h1_rows[0].cpu().numpy(), layer.h1_rows[1].cpu().numpy()
    want = np.zeros((W, bs, h))
    size = np.zeros((W, bs, h))
    for d in range(W):
        for r in range(ep[d, -1]):
            e = d * L + int(np.searchsorted(ep[d], r, side="right")) // W
            s, t, k = assist[d, r]
            assert ids[s, t, k] == e
            g, u = gq[e] @ xq[s, t] * gs[e] * xs[s, t], uq[e] @ xq[s, t] * us[e] * xs[s, t]
            act = g / (1 + np.exp(-g)) * u
            # whole sums, three roundings with the scales each, the fast functions, one rounding to bf16
            assert (np.abs(h1[d, r] - act) <= (2.0 ** -8 + 2.0 ** -16 + 8 * EPS) * np.abs(act) + 8 * EPS * np.abs(u)).all()
            q, sc = int8(layer.h1[d, r][None])
            assert np.array_equal(codes[d, r], q[0]) and scales[d, r] == sc[0]
            z = dq[e] @ codes[d, r].astype(np.float64) * ds[e] * float(scales[d, r])
            assert (np.abs(y[d, r] - z) <= (2.0 ** -8 + 3 * EPS) * np.abs(z)).all()
            want[s, t] += weights[s, t, k] * y[d, r]
            size[s, t] += np.abs(weights[s, t, k] * y[d, r])
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (K + 1) * 2 * EPS * size).all()


def test_layer_near_the_bf16_layer():
    """8-bit rounding with a scale a row is off by at most half a step, 1/254 of the row's largest magnitude, some 1/250 of
    4 standard deviations: each of rows, weights and the intermediate by 0.005 of its size in the mean square (a
    uniform rounding's sqrt(1/12) of 4/127), the sums of gate, up and down by less than twice that each."""
    layer, x, logits, (wg, wu, wd) = make(W=2, bs=32, h=512, E=8, K=2, I=256, router=dict(score_func=M.SCORE_SIGMOID))
    out = layer(x, logits)
    cfg = M.config(2, 32, 512, 2, 8, torch.bfloat16, ffn_intermediate=256)
    ws = M.alloc_workspace(cfg)
    want = torch.empty_like(x)
    M.dispatch_ffn_combine(cfg, x, layer.ids, None, layer.weights, wg, wu, wd, want, ws)
    assert M.get_device_status(ws) == 0 and M.get_device_status(layer.ws) == 0
    assert float((out.float() - want.float()).norm() / want.float().norm()) < 0.05


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


@pytest.mark.parametrize("kind", ["int8", "mxfp4"])
def test_router_gradient_of_a_step(kind):
    """From the output's gradient to the logits': through the combine, then the router."""
    layer, x, logits, _ = make(seed=4, router=dict(renormalize=False), kind=Int8Layer if kind == "int8" else Mxfp4Layer)
    layer(x, logits)
    grad_out = torch.randn(x.shape, device="cuda").bfloat16()
    gw = layer.weights_gradient(grad_out)
    got = layer.logits_gradient(logits, gw).double().cpu().numpy()
    assert M.get_device_status(layer.ws) == 0
    W, bs, h = x.shape
    K = layer.ids.shape[-1]
    y, g = layer.y.double().cpu().numpy(), grad_out.double().cpu().numpy()
    want = np.zeros((W, bs, K))
    size = np.zeros((W, bs, K))
    ep, assist = layer.rows["ep_recv_count"].cpu().numpy(), layer.rows["assist_info"].cpu().numpy()
    for d in range(W):
        for r in range(ep[d, -1]):
            s, t, k = assist[d, r]
            want[s, t, k], size[s, t, k] = (g[s, t] * y[d, r]).sum(), np.abs(g[s, t] * y[d, r]).sum()
    assert (np.abs(gw.double().cpu().numpy() - want) <= 32 * EPS * size).all()
    ids, lg = layer.ids.cpu().numpy().reshape(-1, K), logits.double().cpu().numpy()
    for t in range(W * bs):
        d = P.route_gradient(lg[t], ids[t], want.reshape(-1, K)[t], False, False, 1.0)
        assert np.allclose(got[t], d, rtol=0, atol=2.0 ** -17 * (np.abs(want.reshape(-1, K)[t]).max() + size.reshape(-1, K)[t].max()))
