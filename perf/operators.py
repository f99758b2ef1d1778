"""The operators around the experts, as cases to measure: routing with its
gradient, microscaled 4-bit (MX FP4) quantisation, and the grouped product of
dispatched MX FP4 rows with every expert's MX FP4 weights.

Where ``own`` is false, ``run`` computes an operator in its plain form:
elementary torch operations in 32 bits, rounded once at the end. Where it is
true, ``run`` makes the framework's own calls. ``exact`` holds the definitions
in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the eight magnitudes of the 4-bit format
BLOCK = 32        # elements that share one E8M0 scale
NEAR_TIE = 1e-6   # keys nearer than this (but not equal) leave the choice to the last bits: such tokens are drawn again


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of a serving loop: only latency counts
        dict(name="route_one_token", op="route", tokens=1, experts=256, topk=8, groups=8, topk_group=4, score="sigmoid",
             bias=True, renormalize=True, scaling=2.5, dtype="f32", masked=0),
        # the decode layer's step (8 ranks x 64 tokens): softmax over half-width logits
        dict(name="route_decode", op="route", tokens=512, experts=128, topk=8, groups=1, topk_group=1, score="softmax",
             bias=False, renormalize=True, scaling=1.0, dtype="bf16", masked=0),
        # a prefill or training batch of odd length, a few experts masked out
        dict(name="route_prefill", op="route", tokens=65521, experts=256, topk=8, groups=8, topk_group=4, score="sigmoid",
             bias=True, renormalize=True, scaling=2.5, dtype="f32", masked=3),
        # the gradient at the decode layer's batch: only the chosen experts' logits get one
        dict(name="route_grad_renormalized", op="route_grad", tokens=4096, experts=256, topk=8, score="sigmoid",
             renormalize=True, scaling=2.5, dtype="bf16"),
        # a training batch whose weights keep the softmax over all experts: every logit gets a gradient
        dict(name="route_grad_softmax", op="route_grad", tokens=65536, experts=256, topk=8, score="softmax",
             renormalize=False, scaling=1.0, dtype="f32"),
        # activations of the decode layer, scales a row after the other as dispatch writes them
        dict(name="quantize_rows", op="quantize", experts=1, rows=512, cols=2048, dtype="bf16", layout="rows"),
        # weights of 128 experts (gate and up, 2048 -> 2 x 512), scales laid out for the product
        dict(name="quantize_weights", op="quantize", experts=128, rows=1024, cols=2048, dtype="bf16", layout="tiled"),
        # one active token in 8 ranks: 8 rows, each with an expert of its own
        dict(name="product_one_token", op="product", ranks=8, bs=1, one_token=True, experts=128, topk=8, k=2048, n=1024,
             swiglu=True, out="bf16", skew=0.0),
        # the decode layer's gate and up: weights streamed once for a few rows an expert
        dict(name="product_decode_gate_up", op="product", ranks=8, bs=64, one_token=False, experts=128, topk=8, k=2048,
             n=1024, swiglu=True, out="bf16", skew=0.0),
        # the decode layer's down projection
        dict(name="product_decode_down", op="product", ranks=8, bs=64, one_token=False, experts=128, topk=8, k=512, n=2048,
             swiglu=False, out="bf16", skew=0.0),
        # the large benchmark batch (16 ranks x 256 tokens, hidden 7168), some experts asked for far more often than others
        dict(name="product_wide_gate_up", op="product", ranks=16, bs=256, one_token=False, experts=256, topk=8, k=7168,
             n=1024, swiglu=True, out="bf16", skew=0.5),
        # prefill: about a thousand rows an expert
        dict(name="product_prefill_gate_up", op="product", ranks=8, bs=2048, one_token=False, experts=128, topk=8, k=2048,
             n=1024, swiglu=True, out="bf16", skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_grad", "quantize", "product"))
    if op in ("route", "route_grad"):
        group_size = _log_int(rng, 1, 64)
        groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
        experts = max(2, min(512, group_size * groups if groups > 1 else _log_int(rng, 4, 512)))
        if experts % groups:
            groups = 1
        topk_group = rng.randint(1, groups)
        topk = rng.randint(1, min(16, topk_group * (experts // groups)))
        case = dict(op=op, tokens=min(_log_int(rng, 1, 65536), 65536 * 256 // experts), experts=experts, topk=topk,
                    score=rng.choice(("softmax", "sigmoid")), renormalize=rng.random() < 0.6,
                    scaling=rng.choice((1.0, 2.5)), dtype=rng.choice(("f32", "bf16", "f16")))
        if op == "route_grad" and topk == 1:
            case["renormalize"] = False  # one renormalised weight is constant: nothing to learn from
        if op == "route":
            case.update(groups=groups, topk_group=topk_group, bias=rng.random() < 0.5, masked=rng.choice((0, 0, 1)))
        return case
    if op == "quantize":
        cols = 2 * _log_int(rng, 8, 3584)
        layout = rng.choice(("rows", "tiled"))
        experts = _log_int(rng, 1, 64) if layout == "tiled" else 1
        rows = max(1, min(_log_int(rng, 1, 65536), (1 << 27) // (cols * experts)))
        return dict(op=op, experts=experts, rows=rows, cols=cols, dtype=rng.choice(("f32", "bf16", "f16")), layout=layout)
    ranks = rng.choice((2, 4, 8))
    experts = ranks * _log_int(rng, 1, 16)
    topk = rng.randint(1, min(8, experts))
    k = BLOCK * _log_int(rng, 2, 128)
    swiglu = rng.random() < 0.5
    n = 2 * _log_int(rng, 16, 1024) if swiglu else _log_int(rng, 16, 2048)
    bs = min(_log_int(rng, 1, 512), max(1, (1 << 37) // (ranks * topk * k * n)))
    return dict(op=op, ranks=ranks, bs=bs, one_token=False, experts=experts, topk=topk, k=k, n=n, swiglu=swiglu,
                out=rng.choice(("bf16", "f16")), skew=rng.choice((0.0, 0.5)))


# ------------------------------------------------------------------ the inputs

def _generator(seed, salt):
    return torch.Generator(device="cuda").manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)


def _near_ties(c, logits, bias):
    """The tokens whose choice of groups or experts hangs on the last bits of a 32-bit key, or None where keys are the logits themselves."""
    top2 = c.get("groups", 1) > 1
    if bias is None and not top2:
        return None
    x = logits.double()
    key = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    key = torch.where(torch.isinf(x), -torch.inf, key + (0.0 if bias is None else bias.double()))
    near = torch.zeros(x.shape[0], dtype=torch.bool, device=x.device)
    if top2:
        g = key.view(x.shape[0], c["groups"], -1)
        best = g.topk(min(2, g.shape[-1]), -1).values
        value = torch.where(torch.isinf(best), 0.0, best).sum(-1)
        value = torch.where(torch.isinf(best[..., 0]), -torch.inf, value)
        order = value.sort(-1, descending=True).values
        if c["topk_group"] < c["groups"]:
            gap = order[:, c["topk_group"] - 1] - order[:, c["topk_group"]]
            near |= gap < NEAR_TIE
        chosen = value >= order[:, c["topk_group"] - 1 : c["topk_group"]]
        key = torch.where(chosen[..., None], g, -torch.inf).view_as(key)
    best = key.topk(min(c["topk"] + 1, key.shape[-1]), -1).values
    gap = best[:, :-1] - best[:, 1:]
    return near | ((gap < NEAR_TIE) & (gap != 0)).any(-1)


def _logits(c, g):
    return (torch.randn(c["tokens"], c["experts"], generator=g, device="cuda") * 1.5).to(DTYPES[c["dtype"]])


def _prepare_route(c, seed):
    g = _generator(seed, 1)
    # the balancing bias moves in steps of a thousandth
    bias = torch.randint(-50, 51, (c["experts"],), generator=g, device="cuda").float() * 1e-3 if c["bias"] else None
    out = torch.randperm(c["experts"], generator=g, device="cuda")[: c["masked"]]
    logits = _logits(c, g)
    logits[:, out] = -torch.inf
    for _ in range(12):
        near = _near_ties(c, logits, bias)
        if near is None or not bool(near.any()):
            break
        other = _logits(c, g)
        other[:, out] = -torch.inf
        logits = torch.where(near[:, None], other, logits)
    T, K = c["tokens"], c["topk"]
    return dict(case=c, logits=logits, bias=bias, ids=torch.empty(T, K, dtype=torch.int32, device="cuda"),
                weights=torch.empty(T, K, dtype=torch.float32, device="cuda"))


def _prepare_route_grad(c, seed):
    g = _generator(seed, 2)
    logits = _logits(c, g)
    ids = logits.float().topk(c["topk"], -1).indices.int().contiguous()  # what routing chose
    grad = torch.randn(c["tokens"], c["topk"], generator=g, device="cuda")
    return dict(case=c, logits=logits, ids=ids, grad=grad, grad_logits=torch.empty_like(logits))


def _prepare_quantize(c, seed):
    g = _generator(seed, 3)
    x = torch.empty(c["experts"], c["rows"], c["cols"], dtype=DTYPES[c["dtype"]], device="cuda")
    for e in range(c["experts"]):
        x[e] = torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * (0.02 if c["layout"] == "tiled" else 1.0)
    blocks = -(-c["cols"] // BLOCK)
    if c["layout"] == "rows":
        scales = torch.zeros(c["experts"], c["rows"], blocks, dtype=torch.uint8, device="cuda")
    else:
        scales = torch.zeros(c["experts"], -(-c["rows"] // 128), -(-blocks // 4), 512, dtype=torch.uint8, device="cuda")
    codes = torch.zeros(c["experts"], c["rows"], c["cols"] // 2, dtype=torch.uint8, device="cuda")
    return dict(case=c, x=x, codes=codes, scales=scales)


def _receive_counts(c, g):
    """Rows of every (expert, source rank) segment of a routed batch, as dispatch would count them."""
    W, E, T = c["ranks"], c["experts"], c["ranks"] * c["bs"]
    popular = torch.log(torch.arange(1, E + 1, device="cuda").double()) * -c["skew"]
    popular = popular[torch.randperm(E, generator=g, device="cuda")]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda", dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
    ids = (popular + noise).topk(c["topk"], -1).indices
    source = torch.arange(T, device="cuda") // c["bs"]
    if c["one_token"]:
        ids, source = ids[:1], source[:1]
    return torch.bincount((ids * W + source[:, None]).reshape(-1), minlength=E * W).view(E, W)


def _prepare_product(c, seed):
    g = _generator(seed, 4)
    W, E, K, N = c["ranks"], c["experts"], c["k"], c["n"]
    L = E // W
    A = c["bs"] * W * min(L, c["topk"])  # rows that a rank has room for
    segments = _receive_counts(c, g)
    ep = segments.view(W, L * W).cumsum(-1).int().contiguous()
    count = segments.sum(-1)
    first = torch.arange(E, device="cuda") // L * A + (count.view(W, L).cumsum(-1) - count.view(W, L)).view(-1)
    # the plan of the plain form: the experts that have rows, and each one's rows, padded to the longest
    experts = count.nonzero()[:, 0]
    place = torch.arange(int(count.max()), device="cuda")
    slots = torch.where(place < count[experts, None], first[experts, None] + place, W * A)
    used = slots.view(-1) < W * A
    rows = slots.view(-1)[used]
    x = torch.zeros(W * A, K // 2, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(W * A, K // BLOCK, dtype=torch.uint8, device="cuda")
    x[rows], xs[rows] = _to_mx(torch.randn(rows.numel(), K, generator=g, device="cuda"))
    w = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w[e], ws[e] = _to_mx(torch.randn(N, K, generator=g, device="cuda") * 0.02)
    cols = N // 2 if c["swiglu"] else N
    y = torch.zeros(W, A, cols, dtype=DTYPES[c["out"]], device="cuda")
    return dict(case=c, x=x.view(W, A, -1), x_scales=xs.view(W, A, -1), ep_recv_count=ep, w=w, w_scales=_tile(ws), y=y,
                experts=experts, rows=rows, at=used.nonzero()[:, 0], padded=slots.numel())


def prepare(case, seed):
    return {"route": _prepare_route, "route_grad": _prepare_route_grad, "quantize": _prepare_quantize,
            "product": _prepare_product}[case["op"]](case, seed)


# ------------------------------------------------------------------ the plain forms

def _scores(x, kind):
    """Scores of 32-bit logits; an expert whose logit is -inf or no number is masked out and scores 0."""
    masked = torch.isnan(x) | (x == -torch.inf)
    if kind == "sigmoid":
        return torch.where(masked, 0.0, 1.0 / (1.0 + torch.exp(-x))), masked
    x = torch.where(masked, -torch.inf, x)
    top = x.amax(-1, keepdim=True)
    e = torch.where(masked, 0.0, torch.where(x == top, 1.0, torch.exp(x - top)))
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), masked


def _weights(picked, c):
    if c["renormalize"]:
        total = picked.sum(-1, keepdim=True)
        picked = torch.where(total > 0, picked / total, 0.0)
    return picked * c["scaling"]


def _route_plain(s):
    c, x = s["case"], s["logits"].float()
    scores, masked = _scores(x, c["score"])
    top2 = c["groups"] > 1
    key = x if s["bias"] is None and not top2 else scores if s["bias"] is None else scores + s["bias"]
    key = torch.where(masked | torch.isnan(key), -torch.inf, key) + 0.0
    order = key.sort(dim=-1, descending=True, stable=True).indices
    if top2:
        T, G = x.shape[0], c["groups"]
        best = key.view(T, G, -1).sort(-1, descending=True).values[..., :2]
        value = torch.where(best == -torch.inf, 0.0, best).sum(-1)
        value = torch.where(best[..., 0] == -torch.inf, -torch.inf, value)
        chosen = torch.zeros(T, G, dtype=torch.int32, device=x.device)
        chosen.scatter_(1, value.sort(dim=-1, descending=True, stable=True).indices[:, : c["topk_group"]], 1)
        inside = chosen.repeat_interleave(x.shape[1] // G, 1).gather(1, order)
        order = order.gather(1, inside.sort(dim=-1, descending=True, stable=True).indices)
    ids = order[:, : c["topk"]]
    s["ids"].copy_(ids)
    s["weights"].copy_(_weights(scores.gather(1, ids), c))
    return {"ids": s["ids"], "weights": s["weights"]}


def _route_grad_plain(s):
    c, x, ids = s["case"], s["logits"].float(), s["ids"].long()
    grad = s["grad"] * c["scaling"]
    scores, _ = _scores(x, c["score"])
    picked = scores.gather(1, ids)
    if c["renormalize"]:
        total = picked.sum(-1, keepdim=True)
        share = torch.where(total > 0, picked / total, 0.0)
        mean = (grad * share).sum(-1, keepdim=True)
        # softmax: the shares are a softmax over the chosen logits
        local = share * (grad - mean)
        local = local if c["score"] == "softmax" else local * (1.0 - picked)
    else:
        local = grad * picked if c["score"] == "softmax" else grad * picked * (1.0 - picked)
    out = torch.zeros_like(x).scatter_(1, ids, local)
    if c["score"] == "softmax" and not c["renormalize"]:
        out -= scores * local.sum(-1, keepdim=True)
    s["grad_logits"].copy_(out)
    return {"grad_logits": s["grad_logits"]}


def _power_of_two(e):
    """2^e in 32 bits for whole e in [-127, 127], from the bits."""
    return torch.where(e >= -126, (e + 127) << 23, 0x00400000).int().view(torch.float32)


def _to_mx(x):
    """Packed E2M1 codes and E8M0 bytes of the last axis, 32 elements a scale."""
    shape, cols = x.shape[:-1], x.shape[-1]
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(*shape, blocks, BLOCK)
    amax = v.abs().amax(-1)
    # floor(log2 amax) - 2: the largest magnitude is 1.5 * 2^2
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    m = v.abs() * _power_of_two(-exponent)[..., None]
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).byte()
    code = (code + 8 * torch.signbit(v).byte()).view(*shape, blocks * BLOCK)[..., :cols]
    return code[..., 0::2] + 16 * code[..., 1::2], (exponent + 127).byte()


def _tile(scales):
    """Scales [E, N, blocks] in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 + (r // 32) * 4 + b of a tile, zeros beyond the edges."""
    E, N, B = scales.shape
    nt, bt = -(-N // 128), -(-B // 4)
    s = torch.nn.functional.pad(scales, (0, bt * 4 - B, 0, nt * 128 - N)).view(E, nt, 4, 32, bt, 4)
    return s.permute(0, 1, 4, 3, 2, 5).reshape(E, nt, bt, 512)


def _untile(tiles, N, B):
    E, nt, bt, _ = tiles.shape
    return tiles.view(E, nt, bt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, nt * 128, bt * 4)[:, :N, :B]


def _quantize_plain(s):
    codes, scales = _to_mx(s["x"])
    s["codes"].copy_(codes)
    s["scales"].copy_(scales if s["case"]["layout"] == "rows" else _tile(scales))
    return {"codes": s["codes"], "scales": s["scales"]}


def _from_mx(codes, scales):
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack((value[byte & 15], value[byte >> 4]), -1)
    v = pair[codes.int()].flatten(-2)
    return (v.view(*scales.shape, BLOCK) * _power_of_two(scales.int() - 127)[..., None]).view(v.shape)


def _product_plain(s):
    c = s["case"]
    E, N, half = s["w"].shape
    some = s["experts"]
    x = _from_mx(s["x"].flatten(0, 1)[s["rows"]], s["x_scales"].flatten(0, 1)[s["rows"]])
    w = _from_mx(s["w"][some], _untile(s["w_scales"][some], N, half * 2 // BLOCK))
    padded = torch.zeros(s["padded"], half * 2, device=x.device)
    padded[s["at"]] = x
    y = torch.bmm(padded.view(some.numel(), -1, half * 2), w.transpose(1, 2)).view(-1, N)[s["at"]]
    if c["swiglu"]:  # the even output features are the gates, the odd ones what they gate
        gate, up = y[:, 0::2], y[:, 1::2]
        y = gate / (1.0 + torch.exp(-gate)) * up
    s["y"].flatten(0, 1)[s["rows"]] = y.to(s["y"].dtype)
    return {"y": s["y"]}


# ------------------------------------------------------------------ the framework's calls

def _product_own(s):
    from combine_route_scan_gb300 import moe as M
    if "ws" not in s:  # the configuration and workspace that the program keeps from its dispatch
        c = s["case"]
        s["cfg"] = M.config(c["ranks"], c["bs"], c["k"], c["topk"], c["experts"], torch.bfloat16, quant_mode=4,
                            expand_dtype="fp4_e2m1")
        s["ws"] = M.alloc_workspace(s["cfg"])
    M.expert_product(s["cfg"], s["x"], s["x_scales"], s["ep_recv_count"], s["w"], s["w_scales"], s["y"],
                     epilogue=M.EPI_SWIGLU if s["case"]["swiglu"] else M.EPI_NONE, ws=s["ws"])
    return {"y": s["y"]}


def _router(s):
    from combine_route_scan_gb300 import moe as M
    if "router" not in s:
        c = s["case"]
        groups = c.get("groups", 1)
        s["router"] = M.router_config(c["tokens"], c["experts"], c["topk"], s["logits"].dtype, group_num=groups,
                                      topk_group=c.get("topk_group", 1),
                                      group_score=M.GROUP_TOP2_SUM if groups > 1 else M.GROUP_MAX,
                                      score_func=M.SCORE_SIGMOID if c["score"] == "sigmoid" else M.SCORE_SOFTMAX,
                                      renormalize=c["renormalize"], scaling=c["scaling"])
    return M, s["router"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"route": _route_plain, "route_grad": _route_grad_plain, "quantize": _quantize_plain,
                "product": _product_plain}[op](s)
    if op == "product":
        return _product_own(s)
    if op == "quantize":
        from combine_route_scan_gb300 import moe as M
        M.mx_quantize(s["x"], s["codes"], s["scales"], layout=M.SF_ROWS if s["case"]["layout"] == "rows" else M.SF_TILED)
        return {"codes": s["codes"], "scales": s["scales"]}
    M, router = _router(s)
    if op == "route":
        M.route(router, s["logits"], s["bias"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    M.route_backward(router, s["logits"], s["ids"], s["grad"], s["grad_logits"])
    return {"grad_logits": s["grad_logits"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "route":
        T, E, K = c["tokens"], c["experts"], c["topk"]
        return {"bytes": T * E * size[c["dtype"]] + T * K * 8 + (4 * E if c["bias"] else 0), "flops": 8 * T * E}
    if c["op"] == "route_grad":
        T, E, K = c["tokens"], c["experts"], c["topk"]
        dense = c["score"] == "softmax" and not c["renormalize"]
        read = T * E if dense else T * K  # only the chosen experts' logits are needed where the others cancel
        return {"bytes": (read + T * E) * size[c["dtype"]] + T * K * 8, "flops": T * (8 * E if dense else 8 * K)}
    if c["op"] == "quantize":
        n = c["experts"] * c["rows"] * c["cols"]
        return {"bytes": n * size[c["dtype"]] + n // 2 + n // BLOCK, "flops": 3 * n}
    T = 1 if c["one_token"] else c["ranks"] * c["bs"]
    rows, E, K, N = T * c["topk"], c["experts"], c["k"], c["n"]
    active = E * (1.0 - (1.0 - c["topk"] / E) ** T)  # experts that some row goes to, on average
    row = K / 2 + K / BLOCK
    cols = N // 2 if c["swiglu"] else N
    return {"bytes": active * N * row + rows * (row + cols * size[c["out"]]) + E * c["ranks"] * 4, "flops": 2.0 * rows * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _route_exact(s):
    c, x = s["case"], s["logits"].double()
    K, E = c["topk"], x.shape[1]
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    if s["bias"] is None and c["groups"] == 1:
        key = x
    else:
        key = score if s["bias"] is None else score + s["bias"].double()
    key = key.masked_fill(x == -torch.inf, -torch.inf)
    closed = torch.zeros_like(key, dtype=torch.bool)
    if c["groups"] > 1:
        parts = key.unflatten(1, (c["groups"], E // c["groups"]))
        first = parts.max(-1)
        second = parts.scatter(2, first.indices[..., None], -torch.inf).amax(-1)
        value = first.values + second.masked_fill(second == -torch.inf, 0.0)
        open_ = torch.ones_like(value, dtype=torch.bool)
        for _ in range(c["groups"] - c["topk_group"]):  # drop the worst group, the highest index among equals
            worst = c["groups"] - 1 - value.flip(1).argmin(1)
            open_ = open_.scatter(1, worst[:, None], False)
            value = value.scatter(1, worst[:, None], torch.inf)
        closed = ~open_.repeat_interleave(E // c["groups"], 1)
    picks = []
    index = torch.arange(E, device=x.device)
    taken = closed
    for _ in range(K):  # the largest key left, the lowest index among equals
        best = key.masked_fill(taken, -torch.inf).amax(1, keepdim=True)
        at = torch.where((key == best) & ~taken, index, E).amin(1)
        picks.append(at)
        taken = taken.scatter(1, at[:, None], True)
    w = torch.stack([score.gather(1, p[:, None])[:, 0] for p in picks], 1)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": w * c["scaling"]}


def _route_grad_exact(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    w = score.gather(1, s["ids"].long())
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    (w * c["scaling"] * s["grad"].double()).sum().backward()
    return {"grad_logits": x.grad}


def _values64(codes, scales):
    low, high = codes & 15, codes >> 4
    c = torch.stack((low, high), -1).flatten(-2).int()
    exponent, mantissa = (c >> 1) & 3, c & 1
    v = torch.where(exponent == 0, mantissa * 0.5, (1.0 + 0.5 * mantissa) * torch.exp2((exponent - 1).double()))
    v = torch.where(c & 8 != 0, -v, v).double()
    return v * torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, -1)


def _product_exact(s):
    c = s["case"]
    W, A, _ = s["x"].shape
    L, N, K = c["experts"] // W, c["n"], c["k"]
    ep = s["ep_recv_count"].tolist()
    r = torch.arange(N, device="cuda")
    b = torch.arange(K // BLOCK, device="cuda")
    at = (r[:, None] % 32) * 16 + (r[:, None] % 128) // 32 * 4 + b % 4
    y = torch.zeros(W, A, s["y"].shape[-1], dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        d, le = divmod(e, L)
        lo, hi = ep[d][le * W - 1] if le else 0, ep[d][le * W + W - 1]
        if hi == lo:
            continue
        scales = s["w_scales"][e][r[:, None] // 128, b // 4, at]
        out = _values64(s["x"][d, lo:hi], s["x_scales"][d, lo:hi]) @ _values64(s["w"][e], scales).T
        if c["swiglu"]:
            out = out[:, 0::2] * torch.sigmoid(out[:, 0::2]) * out[:, 1::2]
        y[d, lo:hi] = out
    return {"y": y}


def exact(case, seed):
    if case["op"] == "quantize":
        return None  # codes and scale bytes are whole numbers, fixed by the format to the last bit
    s = prepare(case, seed)
    return {"route": _route_exact, "route_grad": _route_grad_exact, "product": _product_exact}[case["op"]](s)
