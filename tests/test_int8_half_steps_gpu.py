"""moe_int8_quantize takes no quotient by a division but a reciprocal, a product and one correction: its codes next to
every half step, for every scale of a binade, against the division's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    B.build()


def rows_of(mantissas, sign):
    """A row for each largest magnitude 1.m (exponent 0): it, then half a step to 126.5 and two fp32 numbers to either side."""
    amax = (mantissas + 0x3F800000).view(torch.float32)[:, None]
    scale = amax / torch.full_like(amax, 127.0)  # a quotient: by a number torch multiplies by its reciprocal
    half = torch.arange(127, device="cuda", dtype=torch.float64) + 0.5
    near = (half * scale.double()).float()
    near = (near.view(torch.int32)[..., None] + torch.arange(-2, 3, device="cuda", dtype=torch.int32)).view(torch.float32).flatten(1)
    x = torch.zeros(len(mantissas), 640, device="cuda")
    x[:, :1] = amax
    x[:, 1:636] = near
    x[:, 1:636:2] *= sign
    x[:, 2:636:2] *= -sign
    return x, scale


def test_codes_next_to_every_half_step_at_every_scale():
    rows = 1 << 16
    codes, scales = torch.empty(rows, 640, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for n, first in enumerate(range(0, 1 << 23, rows)):
        x, scale = rows_of(torch.arange(first, first + rows, device="cuda", dtype=torch.int32), 1 - 2 * (n % 2))
        M.int8_quantize(x, codes, scales)
        want = torch.round(x / scale)
        wrong += (codes != want).sum() + (scales != scale[:, 0]).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("exponent", [-93, -60, 40, 120])
def test_the_same_far_from_one(exponent):
    """The scales' mantissas by random, the magnitudes from where the smallest residuals are still normal numbers on."""
    g = torch.Generator(device="cuda").manual_seed(exponent + 200)
    x, _ = rows_of(torch.randint(0, 1 << 23, (1 << 15,), generator=g, device="cuda", dtype=torch.int32), 1)
    x = x * 2.0 ** exponent  # exact
    codes, scales = M.alloc_int8(x)
    M.int8_quantize(x, codes, scales)
    scale = x[:, :1] / torch.full_like(x[:, :1], 127.0)
    assert torch.equal(scales, scale[:, 0])
    assert torch.equal(codes.float(), torch.round(x / scale))
