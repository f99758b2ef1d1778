"""More operators around the experts, as cases to measure: rows quantised to 8-bit
integers with a scale each, the grouped product of dispatched int8 rows with every
expert's int8 weights (scales for each row and output channel), and the gradients
of combine and dispatch (rows sorted by expert and back, with their weights).

Where ``own`` is false, ``run`` computes an operator in its plain form:
elementary torch operations in 32 bits, rounded once at the end. Where it is
true, ``run`` makes the framework's own calls. ``exact`` holds the definitions
in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # activations of the decode layer between its two products (8 ranks x 64 tokens, intermediate 512): only the
        # rows that were received
        dict(name="quantize_decode_rows", op="quantize", ranks=8, bs=64, experts=128, topk=8, cols=512, dtype="bf16",
             received=True),
        # weights of 128 experts (gate and up, 2048 -> 2 x 512): one scale for each output channel
        dict(name="quantize_weights", op="quantize", ranks=128, bs=1024, experts=128, topk=1, cols=2048, dtype="bf16",
             received=False),
        # one active token in 8 ranks: 8 rows, each with an expert of its own
        dict(name="product_one_token", op="product", ranks=8, bs=1, one_token=True, experts=128, topk=8, k=2048, n=1024,
             swiglu=True, out="bf16", skew=0.0),
        # the decode layer's gate and up: weights streamed once for a few rows an expert
        dict(name="product_decode_gate_up", op="product", ranks=8, bs=64, one_token=False, experts=128, topk=8, k=2048,
             n=1024, swiglu=True, out="bf16", skew=0.0),
        # the decode layer's down projection
        dict(name="product_decode_down", op="product", ranks=8, bs=64, one_token=False, experts=128, topk=8, k=512, n=2048,
             swiglu=False, out="f16", skew=0.0),
        # the large benchmark batch (16 ranks x 256 tokens, hidden 7168), some experts asked for far more often than others
        dict(name="product_wide_gate_up", op="product", ranks=16, bs=256, one_token=False, experts=256, topk=8, k=7168,
             n=1024, swiglu=True, out="bf16", skew=0.5),
        # prefill: about a thousand rows an expert
        dict(name="product_prefill_gate_up", op="product", ranks=8, bs=2048, one_token=False, experts=128, topk=8, k=2048,
             n=1024, swiglu=True, out="bf16", skew=0.0),
        # the smallest profiling shape (2 ranks x 8 tokens, hidden 256, top-2): only latency counts
        dict(name="combine_grad_small", op="combine_grad", ranks=2, bs=8, experts=4, topk=2, zero=0, copy=0, mask=0, h=256,
             dtype="f16"),
        # a training step over the benchmark's tokens, experts and hidden size, with special experts and masked picks
        dict(name="combine_grad_train", op="combine_grad", ranks=4, bs=1024, experts=256, topk=8, zero=2, copy=2, mask=2,
             h=7168, dtype="bf16"),
        # fine-tuning on the decode layer's batch, weights applied by the experts' side (their gradient comes back by row)
        dict(name="dispatch_grad_small", op="dispatch_grad", ranks=8, bs=64, experts=128, topk=8, zero=0, copy=0, mask=0,
             h=2048, dtype="f16", residual=False, weights=True),
        # the training step's other end: a token's rows summed onto what came past the experts
        dict(name="dispatch_grad_train", op="dispatch_grad", ranks=4, bs=1024, experts=256, topk=8, zero=2, copy=2, mask=2,
             h=7168, dtype="bf16", residual=True, weights=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "combine_grad", "dispatch_grad"))
    ranks = rng.choice((2, 4, 8))
    experts = ranks * _log_int(rng, 1, 32)
    topk = rng.randint(1, min(8, experts))
    if op == "quantize":
        cols = _log_int(rng, 16, 7168)
        received = rng.random() < 0.5
        most = (1 << 28) // (cols * ranks * (ranks * 8 if received else 1))
        return dict(op=op, ranks=ranks, bs=max(1, min(_log_int(rng, 1, 8192), most)), experts=experts, topk=topk, cols=cols,
                    dtype=rng.choice(("f32", "bf16", "f16")), received=received)
    if op == "product":
        experts = min(experts, ranks * 16)
        topk = min(topk, experts)
        k = 16 * _log_int(rng, 2, 256)
        swiglu = rng.random() < 0.5
        n = 2 * _log_int(rng, 16, 1024) if swiglu else _log_int(rng, 16, 2048)
        bs = min(_log_int(rng, 1, 512), max(1, (1 << 37) // (ranks * topk * k * n)))
        return dict(op=op, ranks=ranks, bs=bs, one_token=False, experts=experts, topk=topk, k=k, n=n, swiglu=swiglu,
                    out=rng.choice(("bf16", "f16")), skew=rng.choice((0.0, 0.5)))
    h = rng.choice((8, 1)) * _log_int(rng, 8, 896)
    most = (1 << 29) // (h * ranks * ranks * min(topk, experts // ranks))  # elements of all ranks' receive buffers
    case = dict(op=op, ranks=ranks, bs=max(1, min(_log_int(rng, 1, 2048), most)), experts=experts, topk=topk,
                zero=rng.choice((0, 0, 1)), copy=rng.choice((0, 0, 2)), mask=rng.choice((0, 1, 2)), h=h,
                dtype=rng.choice(("bf16", "f16")))
    if op == "dispatch_grad":
        case.update(residual=rng.random() < 0.5, weights=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------ the inputs

def _generator(seed, salt):
    return torch.Generator(device="cuda").manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)


def _capacity(c):
    """Rows that a rank has room for."""
    return c["bs"] * c["ranks"] * min(c["experts"] // c["ranks"], c["topk"])


def _choose(c, g):
    """Expert ids [T, topk], distinct in a token; the higher `skew`, the more often the popular ones."""
    T, E = c["ranks"] * c["bs"], c["experts"]
    popular = torch.log(torch.arange(1, E + 1, device="cuda").double()) * -c.get("skew", 0.0)
    popular = popular[torch.randperm(E, generator=g, device="cuda")]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda", dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
    return (popular + noise).topk(c["topk"], -1).indices


def _dispatched(c, ids, routed):
    """What dispatch leaves for the picks `routed` of ids: each rank's rows by expert, then by source rank, token and
    place in the token. Receive counts [W, L*W], each received row's place (flat, in all ranks' buffers) and its pick."""
    W, E, A, K = c["ranks"], c["experts"], _capacity(c), c["topk"]
    L = E // W
    pick = routed.reshape(-1).nonzero()[:, 0]
    e = ids.reshape(-1)[pick]
    segment = e * W + pick // (c["bs"] * K)
    segment, order = segment.sort(stable=True)
    pick = pick[order]
    sizes = torch.bincount(segment, minlength=E * W)
    ep = sizes.view(W, L * W).cumsum(-1)
    first = ep[:, -1].cumsum(0) - ep[:, -1]  # rows of the ranks before
    rank = segment // (W * L)
    rows = rank * A + torch.arange(pick.numel(), device="cuda") - first[rank]
    return ep.int().contiguous(), rows, pick


def _codes(v):
    """Codes and scales of the plain quantiser, for inputs of the product."""
    scale = v.abs().amax(-1, keepdim=True) / 127.0
    return torch.round(v / scale).clamp(-127, 127).to(torch.int8), scale[..., 0]


def _prepare_quantize(c, seed):
    g = _generator(seed, 1)
    if not c["received"]:
        mats, rows = c["ranks"], c["bs"]
        x = torch.empty(mats, rows, c["cols"], dtype=DTYPES[c["dtype"]], device="cuda")
        for m in range(mats):
            x[m] = torch.randn(rows, c["cols"], generator=g, device="cuda") * 0.02
        ep, some = None, None
    else:
        ids = _choose(c, g)
        ep, some, _ = _dispatched(c, ids, torch.ones_like(ids, dtype=torch.bool))
        mats, rows = c["ranks"], _capacity(c)
        x = torch.zeros(mats, rows, c["cols"], dtype=DTYPES[c["dtype"]], device="cuda")
        v = torch.randn(some.numel(), 2, c["cols"], generator=g, device="cuda")
        x.flatten(0, 1)[some] = (torch.nn.functional.silu(v[:, 0]) * v[:, 1]).to(x.dtype)  # what SwiGLU gives
    return dict(case=c, x=x, ep_recv_count=ep, some=some, codes=torch.zeros(x.shape, dtype=torch.int8, device="cuda"),
                scales=torch.zeros(mats, rows, device="cuda"))


def _prepare_product(c, seed):
    g = _generator(seed, 2)
    W, E, K, N, A = c["ranks"], c["experts"], c["k"], c["n"], _capacity(c)
    ids = _choose(c, g)
    routed = torch.ones_like(ids, dtype=torch.bool)
    if c["one_token"]:
        routed[1:] = False
    ep, rows, pick = _dispatched(c, ids, routed)
    x = torch.zeros(W * A, K, dtype=torch.int8, device="cuda")
    xs = torch.zeros(W * A, device="cuda")
    x[rows], xs[rows] = _codes(torch.randn(rows.numel(), K, generator=g, device="cuda"))
    w = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    ws = torch.empty(E, N, device="cuda")
    for e in range(E):
        w[e], ws[e] = _codes(torch.randn(N, K, generator=g, device="cuda") * 0.02)
    # the plan of the plain form: the experts that have rows, and each one's rows padded to the longest
    expert = ids.reshape(-1)[pick]
    count = torch.bincount(expert, minlength=E)
    experts = count.nonzero()[:, 0]
    longest = int(count.max())
    slot = torch.cumsum((count > 0).long(), 0) - 1
    begin = torch.cumsum(count, 0) - count
    at = slot[expert] * longest + torch.arange(rows.numel(), device="cuda") - begin[expert]
    y = torch.zeros(W, A, N // 2 if c["swiglu"] else N, dtype=DTYPES[c["out"]], device="cuda")
    return dict(case=c, x=x.view(W, A, K), x_scales=xs.view(W, A), ep_recv_count=ep, w=w, w_scales=ws, y=y, experts=experts,
                rows=rows, at=at, padded=experts.numel() * longest)


def _picks(c, g):
    """Ids with zero and copy experts among them and a mask, as expert_ids and active_mask take them, and which picks are
    routed to an expert and which copy their token."""
    T, K, E = c["ranks"] * c["bs"], c["topk"], c["experts"]
    ids = _choose(c, g)
    special = c["zero"] + c["copy"]
    if special:
        to = torch.randint(E, E + special, (T, K), generator=g, device="cuda")
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < 0.1, to, ids)
    active = torch.ones(T, K, dtype=torch.bool, device="cuda")
    mask = None
    if c["mask"] == 1:  # each rank's tokens up to some place
        left = torch.randint(0, c["bs"] + 1, (c["ranks"], 1), generator=g, device="cuda")
        mask = (torch.arange(c["bs"], device="cuda") < left).reshape(T)
        active &= mask[:, None]
    elif c["mask"] == 2:
        mask = torch.rand(T, K, generator=g, device="cuda") >= 0.1
        active &= mask
    return ids, None if mask is None else mask.to(torch.uint8), active & (ids < E), active & (ids >= E + c["zero"])


def _prepare_grad(c, seed):
    g = _generator(seed, 3)
    W, bs, K, h, A, dt = c["ranks"], c["bs"], c["topk"], c["h"], _capacity(c), DTYPES[c["dtype"]]
    ids, mask, routed, copied = _picks(c, g)
    ep, rows, pick = _dispatched(c, ids, routed)
    assist = torch.full((W * A, 3), -1, dtype=torch.int32, device="cuda")
    assist[rows] = torch.stack((pick // (bs * K), pick // K % bs, pick % K), -1).int()
    s = dict(case=c, ids=ids.int().view(W, bs, K), mask=mask, ep_recv_count=ep, assist_info=assist.view(W, A, 3), rows=rows,
             pick=pick)
    if c["op"] == "combine_grad":
        y = torch.zeros(W * A, h, dtype=dt, device="cuda")
        y[rows] = torch.randn(rows.numel(), h, generator=g, device="cuda").to(dt)
        weights = torch.rand(W * bs, K, generator=g, device="cuda") + 0.05
        s.update(expert_out=y.view(W, A, h), weights=(weights / weights.sum(-1, keepdim=True)).view(W, bs, K), copied=copied,
                 grad_out=torch.randn(W, bs, h, generator=g, device="cuda").to(dt),
                 x=torch.randn(W, bs, h, generator=g, device="cuda").to(dt) if c["copy"] else None,
                 grad_rows=torch.zeros(W, A, h, dtype=dt, device="cuda"),
                 grad_weights=torch.zeros(W, bs, K, device="cuda"),
                 grad_x=torch.zeros(W, bs, h, dtype=dt, device="cuda") if c["copy"] else None)
    else:
        grad = torch.zeros(W * A, h, dtype=dt, device="cuda")
        grad[rows] = torch.randn(rows.numel(), h, generator=g, device="cuda").to(dt)
        s.update(grad_rows=grad.view(W, A, h),
                 residual=torch.randn(W, bs, h, generator=g, device="cuda").to(dt) if c["residual"] else None,
                 grad_row_weights=torch.randn(W, A, generator=g, device="cuda") if c["weights"] else None,
                 grad_x=torch.zeros(W, bs, h, dtype=dt, device="cuda"),
                 grad_weights=torch.zeros(W, bs, K, device="cuda") if c["weights"] else None)
    return s


def prepare(case, seed):
    return {"quantize": _prepare_quantize, "product": _prepare_product}.get(case["op"], _prepare_grad)(case, seed)


# ------------------------------------------------------------------ the plain forms

def _quantize_plain(s):
    x = s["x"] if s["some"] is None else s["x"].flatten(0, 1)[s["some"]]
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)  # a quotient: by a number torch multiplies by its reciprocal
    codes = torch.where(scale > 0, torch.round(x / scale), 0.0).clamp(-127, 127).to(torch.int8)
    if s["some"] is None:
        s["codes"].copy_(codes)
        s["scales"].copy_(scale[..., 0])
    else:
        s["codes"].flatten(0, 1)[s["some"]] = codes
        s["scales"].view(-1)[s["some"]] = scale[:, 0]
    return {"codes": s["codes"], "scales": s["scales"]}


def _product_plain(s):
    c = s["case"]
    E, N, K = s["w"].shape
    some, rows = s["experts"], s["rows"]
    x = s["x"].flatten(0, 1)[rows].float() * s["x_scales"].view(-1)[rows][:, None]
    w = s["w"][some].float() * s["w_scales"][some][..., None]
    padded = torch.zeros(s["padded"], K, device=x.device)
    padded[s["at"]] = x
    y = torch.bmm(padded.view(some.numel(), -1, K), w.transpose(1, 2)).view(-1, N)[s["at"]]
    if c["swiglu"]:  # the even output features are the gates, the odd ones what they gate
        gate, up = y[:, 0::2], y[:, 1::2]
        y = gate / (1.0 + torch.exp(-gate)) * up
    s["y"].flatten(0, 1)[rows] = y.to(s["y"].dtype)
    return {"y": s["y"]}


def _combine_grad_plain(s):
    c, rows, pick = s["case"], s["rows"], s["pick"]
    K = c["topk"]
    g = s["grad_out"].flatten(0, 1).float()
    weights = s["weights"].flatten()
    mine = g[pick // K]
    s["grad_rows"].flatten(0, 1)[rows] = (weights[pick][:, None] * mine).to(s["grad_rows"].dtype)
    gw = torch.zeros_like(weights)
    gw[pick] = (mine * s["expert_out"].flatten(0, 1)[rows].float()).sum(-1)
    out = {"grad_rows": s["grad_rows"], "grad_weights": s["grad_weights"]}
    if s["x"] is not None:
        own_x = (g * s["x"].flatten(0, 1).float()).sum(-1)
        gw = torch.where(s["copied"].flatten(), own_x.repeat_interleave(K), gw)
        kept = torch.where(s["copied"], s["weights"].flatten(0, 1), 0.0).sum(-1)
        s["grad_x"].flatten(0, 1).copy_(kept[:, None] * g)
        out["grad_x"] = s["grad_x"]
    s["grad_weights"].view(-1).copy_(gw)
    return out


def _dispatch_grad_plain(s):
    c, rows, pick = s["case"], s["rows"], s["pick"]
    T, K, h = c["ranks"] * c["bs"], c["topk"], c["h"]
    by_pick = torch.zeros(T * K, h, device=rows.device)
    by_pick[pick] = s["grad_rows"].flatten(0, 1)[rows].float()
    total = by_pick.view(T, K, h).sum(1)
    if s["residual"] is not None:
        total += s["residual"].flatten(0, 1).float()
    s["grad_x"].flatten(0, 1).copy_(total)
    out = {"grad_x": s["grad_x"]}
    if s["grad_weights"] is not None:
        gw = torch.zeros(T * K, device=rows.device)
        gw[pick] = s["grad_row_weights"].view(-1)[rows]
        s["grad_weights"].view(-1).copy_(gw)
        out["grad_weights"] = s["grad_weights"]
    return out


# ------------------------------------------------------------------ the framework's calls

def _config(s):
    """The configuration and workspace that a program keeps from its dispatch."""
    from combine_route_scan_gb300 import moe as M
    if "ws" not in s:
        c = s["case"]
        if c["op"] == "product":
            s["cfg"] = M.config(c["ranks"], c["bs"], c["k"], c["topk"], c["experts"], torch.bfloat16, quant_mode=2)
        else:
            s["cfg"] = M.config(c["ranks"], c["bs"], c["h"], c["topk"], c["experts"], DTYPES[c["dtype"]],
                                zero_expert_num=c["zero"], copy_expert_num=c["copy"], mask_kind=c["mask"])
        s["ws"] = M.alloc_workspace(s["cfg"])
    return M, s["cfg"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"quantize": _quantize_plain, "product": _product_plain, "combine_grad": _combine_grad_plain,
                "dispatch_grad": _dispatch_grad_plain}[op](s)
    if op == "quantize":
        from combine_route_scan_gb300 import moe as M
        M.int8_quantize(s["x"], s["codes"], s["scales"], ep_recv_count=s["ep_recv_count"])
        return {"codes": s["codes"], "scales": s["scales"]}
    M, cfg = _config(s)
    if op == "product":
        M.expert_product_int8(cfg, s["x"], s["x_scales"], s["ep_recv_count"], s["w"], s["w_scales"], s["y"],
                              epilogue=M.EPI_SWIGLU if s["case"]["swiglu"] else M.EPI_NONE, ws=s["ws"])
        return {"y": s["y"]}
    if op == "combine_grad":
        M.combine_backward(cfg, s["grad_out"], s["expert_out"], s["assist_info"], s["ep_recv_count"], s["ids"], s["weights"],
                           s["mask"], s["x"], s["grad_rows"], s["grad_weights"], s["grad_x"], ws=s["ws"])
        out = {"grad_rows": s["grad_rows"], "grad_weights": s["grad_weights"]}
        return out if s["x"] is None else {**out, "grad_x": s["grad_x"]}
    M.dispatch_backward(cfg, s["grad_rows"], s["assist_info"], s["ep_recv_count"], s["ids"], s["mask"], s["grad_x"],
                        residual=s["residual"], grad_expand_scales=s["grad_row_weights"], grad_scales=s["grad_weights"],
                        ws=s["ws"])
    out = {"grad_x": s["grad_x"]}
    return out if s["grad_weights"] is None else {**out, "grad_weights": s["grad_weights"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "quantize":
        rows = c["ranks"] * c["bs"] * (c["topk"] if c["received"] else 1)
        return {"bytes": rows * (c["cols"] * (SIZE[c["dtype"]] + 1) + 4), "flops": 4 * rows * c["cols"]}
    T = c["ranks"] * c["bs"]
    if c["op"] == "product":
        T = 1 if c["one_token"] else T
        rows, E, K, N = T * c["topk"], c["experts"], c["k"], c["n"]
        active = E * (1.0 - (1.0 - c["topk"] / E) ** T)  # experts that some row goes to, on average
        cols = N // 2 if c["swiglu"] else N
        return {"bytes": active * N * (K + 4) + rows * (K + 4 + cols * SIZE[c["out"]]) + E * c["ranks"] * 4,
                "flops": 2.0 * rows * N * K}
    # shares of the picks that go to an expert, and that copy their token
    active = {0: 1.0, 1: 0.5, 2: 0.9}[c["mask"]]
    special = 0.1 if c["zero"] + c["copy"] else 0.0
    rows = T * c["topk"] * active * (1.0 - special)
    copies = T * c["topk"] * active * special * c["copy"] / max(1, c["zero"] + c["copy"])
    row, picks = c["h"] * SIZE[c["dtype"]], T * c["topk"]
    meta = picks * 4 + rows * 12 + c["experts"] * c["ranks"] * 4 + (T if c["mask"] == 1 else picks if c["mask"] == 2 else 0)
    if c["op"] == "combine_grad":
        copying = T * (1.0 - (1.0 - copies / picks) ** c["topk"])  # tokens with a copy
        return {"bytes": T * row + 2 * rows * row + copying * row + (T * row if c["copy"] else 0) + meta + picks * 8,
                "flops": (3 * rows + 2 * copies) * c["h"]}
    return {"bytes": rows * row + T * row * (2 if c["residual"] else 1) + meta + (rows * 4 + picks * 4 if c["weights"] else 0),
            "flops": (rows + (T if c["residual"] else 0)) * c["h"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _received(s):
    """(flat row, expert) of every received row, in order, from the receive counts alone."""
    c = s["case"]
    W, L, A = c["ranks"], c["experts"] // c["ranks"], _capacity(c)
    rows, experts = [], []
    for d, counts in enumerate(s["ep_recv_count"].tolist()):
        for le in range(L):
            lo, hi = counts[le * W - 1] if le else 0, counts[le * W + W - 1]
            rows.append(torch.arange(d * A + lo, d * A + hi, device="cuda"))
            experts.append(d * L + le)
    return rows, experts


def _quantize_exact(s):
    amax = s["x"].double().abs().amax(-1)
    if s["case"]["received"]:
        here = torch.arange(amax.shape[1], device="cuda") < s["ep_recv_count"][:, -1:]
        amax = torch.where(here, amax, 0.0)
    return {"codes": None, "scales": amax / 127}


def _product_exact(s):
    y = torch.zeros(s["y"].flatten(0, 1).shape, dtype=torch.float64, device="cuda")
    x, xs = s["x"].flatten(0, 1), s["x_scales"].view(-1)
    for rows, e in zip(*_received(s)):
        if rows.numel() == 0:
            continue
        z = x[rows].double() @ s["w"][e].double().T
        z = z * xs[rows].double()[:, None] * s["w_scales"][e].double()
        if s["case"]["swiglu"]:
            z = z[:, 0::2] * torch.sigmoid(z[:, 0::2]) * z[:, 1::2]
        y[rows] = z
    return {"y": y.view(s["y"].shape)}


def _grad_exact(s):
    """By each received row's own note of where it came from, and for copies by the tokens' ids."""
    c = s["case"]
    W, bs, K, h, A = c["ranks"], c["bs"], c["topk"], c["h"], _capacity(c)
    combine = c["op"] == "combine_grad"
    gx = None if combine and s["x"] is None else torch.zeros(W, bs, h, dtype=torch.float64, device="cuda")
    gw = torch.zeros(W, bs, K, dtype=torch.float64, device="cuda")
    grad_rows = torch.zeros(W, A, h, dtype=torch.float64, device="cuda") if combine else None
    if not combine and s["residual"] is not None:
        gx += s["residual"].double()
    for rows, _ in zip(*_received(s)):
        if rows.numel() == 0:
            continue
        d, r = rows // A, rows % A
        source, token, place = s["assist_info"][d, r].long().unbind(-1)
        if combine:
            g = s["grad_out"][source, token].double()
            grad_rows[d, r] = s["weights"][source, token, place].double()[:, None] * g
            gw[source, token, place] = torch.einsum("rh,rh->r", g, s["expert_out"][d, r].double())
        else:
            gx.index_put_((source, token), s["grad_rows"][d, r].double(), accumulate=True)
            if s["grad_weights"] is not None:
                gw[source, token, place] = s["grad_row_weights"][d, r].double()
    if not combine:
        return {"grad_x": gx} if s["grad_weights"] is None else {"grad_x": gx, "grad_weights": gw}
    if s["x"] is None:
        return {"grad_rows": grad_rows, "grad_weights": gw}
    for k in range(K):
        copies = s["ids"][..., k] >= c["experts"] + c["zero"]
        if c["mask"] == 1:
            copies &= s["mask"].view(W, bs) != 0
        elif c["mask"] == 2:
            copies &= s["mask"].view(W, bs, K)[..., k] != 0
        source, token = copies.nonzero().unbind(-1)
        g = s["grad_out"][source, token].double()
        gx[source, token] += s["weights"][source, token, k].double()[:, None] * g
        gw[source, token, k] = (g * s["x"][source, token].double()).sum(-1)
    return {"grad_rows": grad_rows, "grad_weights": gw, "grad_x": gx}


def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _quantize_exact, "product": _product_exact}.get(case["op"], _grad_exact)(s)
