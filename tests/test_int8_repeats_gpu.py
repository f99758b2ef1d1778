"""The int8 product on a large skewed batch (16 ranks x 256 tokens of hidden 7168, 256 experts of which some have far more
rows): the same bytes call after call, with other calls between them and beside them, and the 64-bit result rounded once."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()

W, BS, K, E, H, N = 16, 256, 8, 256, 7168, 1024
EPS = 2.0 ** -24


class Batch:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        L = E // W
        popular = torch.log(torch.arange(1, E + 1, device="cuda").double())[torch.randperm(E, generator=g, device="cuda")] * -0.5
        noise = -torch.log(-torch.log(torch.rand(W * BS, E, generator=g, device="cuda", dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
        ids = (popular + noise).topk(K, -1).indices
        source = (torch.arange(W * BS, device="cuda") // BS)[:, None]
        sizes = torch.bincount((ids * W + source).flatten(), minlength=E * W)
        self.ep = sizes.view(W, L * W).cumsum(-1).int().contiguous()
        self.cfg = M.config(W, BS, H, K, E, torch.bfloat16, quant_mode=2)
        self.A = M.workspace_size(self.cfg)[1]
        most = int(self.ep[:, -1].max())
        self.x = torch.zeros(W, self.A, H, dtype=torch.int8, device="cuda")
        self.x[:, :most] = (torch.randn(W, most, H, generator=g, device="cuda") * 30).round().clamp(-127, 127).to(torch.int8)
        self.xs = torch.rand(W, self.A, generator=g, device="cuda") + 0.5
        self.y = torch.empty(W, self.A, N, dtype=torch.bfloat16, device="cuda")

    def run(self, w, ws, space):
        M.expert_product_int8(self.cfg, self.x, self.xs, self.ep, w, ws, self.y, ws=space)


def test_the_same_bytes_and_the_rounded_result():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(E, N, H, dtype=torch.int8, device="cuda")
    for e in range(E):
        w[e] = (torch.randn(N, H, generator=g, device="cuda") * 30).round().clamp(-127, 127).to(torch.int8)
    ws = (torch.rand(E, N, generator=g, device="cuda") + 0.5) / 76000
    a, b = Batch(2), Batch(3)
    space = M.alloc_workspace(a.cfg)
    a.y.fill_(777.0)
    a.run(w, ws, space)
    first = a.y.clone()
    side, beside = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for n in range(8):
        a.y.fill_(777.0)
        b.run(w, ws, space)
        with torch.cuda.stream(side):  # other work on the SMs
            beside @ beside
        a.run(w, ws, space)
        assert torch.equal(a.y, first), n
    assert M.get_device_status(space) == 0
    L, ep = E // W, a.ep.cpu()
    for d in range(W):
        for le in range(L):
            lo, hi = int(ep[d, le * W - 1]) if le else 0, int(ep[d, le * W + W - 1])
            x, v = a.x[d, lo:hi].float(), w[d * L + le].float().T
            # whole numbers whose partial sums are below 2^24 in any order: exact in fp32
            assert lo == hi or float((x.abs() @ v.abs()).max()) < 2 ** 24 - 2 ** 16
            want = (x @ v).double()
            want = want * a.xs[d, lo:hi, None].double() * ws[d * L + le].double()
            # two products in fp32, then one rounding: between the roundings of what is two half steps below and above
            low, high = ((want * (1 + s * 2.01 * EPS)).to(torch.bfloat16).float() for s in (-1, 1))
            got = first[d, lo:hi].float()
            assert bool(((got >= torch.minimum(low, high)) & (got <= torch.maximum(low, high))).all()), (d, le)
        assert bool((first[d, int(ep[d, -1]):] == 777.0).all())
