"""include/moe_experts.h without a GPU: the library exports what it declares,
the configuration's layout matches, sizes and host-side refusals."""
import ctypes
import os
import re

import numpy as np
import pytest

import experts_plain as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from combine_route_scan_gb300 import build
    build.build()
    from combine_route_scan_gb300 import moe
    return moe


def test_library_exports_the_declared_entries(lib):
    with open(os.path.join(ROOT, "include", "moe_experts.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:moe_status_t|uint64_t)\s+(moe_\w+)\s*\(", text, flags=re.M))
    assert names == set(lib.EXPERTS_EXPORTS)
    for name in names:
        assert hasattr(lib.lib(), name), name


def test_router_config_layout(lib):
    assert ctypes.sizeof(lib.RouterConfig) == 48
    assert lib.RouterConfig.scaling.offset == 36
    assert lib.RouterConfig.logits_stride.offset == 40


@pytest.mark.parametrize("experts,rows,cols", [(1, 1, 2), (3, 128, 128), (2, 129, 130), (4, 64, 2048), (0, 5, 32), (5, 0, 32)])
def test_scale_bytes(lib, experts, rows, cols):
    s = np.zeros((experts, rows, -(-cols // 32)), dtype=np.uint8)
    assert lib.mx_scale_bytes(experts, rows, cols, lib.SF_ROWS) == s.size
    assert lib.mx_scale_bytes(experts, rows, cols, lib.SF_TILED) == P.tile_scales(s).size


@pytest.mark.parametrize("args", [(-1, 1, 32, 0), (1, -1, 32, 0), (1, 1, 31, 0), (1, 1, 0, 0), (1, 1, 32, 2), (2, 1 << 30, 32, 0)])
def test_scale_bytes_of_refused_sizes(lib, args):
    assert lib.mx_scale_bytes(*args) == 0


def test_refusals_without_a_gpu(lib):
    L = lib.lib()
    import torch
    rc = lib.router_config(4, 64, 8, torch.float32)
    assert L.moe_route(ctypes.byref(rc), None, None, None, None, None) == 1
    assert L.moe_route(None, None, None, None, None, None) == 1
    assert L.moe_route_backward(ctypes.byref(rc), None, None, None, None, 64, None) == 1
    assert L.moe_mx_quantize(None, 3, 1, 1, 32, 32, 0, 0, None, None, None) == 1
    assert L.moe_mx_quantize(None, 0, 1, 1, 32, 32, 0, 0, None, None, None) == 1  # int32 is no input type
    cfg = lib.config(2, 4, 64, 2, 4, torch.bfloat16)
    for n, k, epi, y, want in ((0, 64, 0, 2, 1), (64, 0, 0, 2, 1), (64, 48, 0, 2, 2), (63, 64, 1, 2, 1), (64, 64, 2, 2, 1),
                               (64, 64, 0, 0, 1), (63, 64, 0, 4, 1)):
        assert L.moe_expert_product(ctypes.byref(cfg), None, None, None, None, None, n, k, epi, y, None, None, None, 0, None) == want
    cfg.topk = 0
    assert L.moe_expert_product(ctypes.byref(cfg), None, None, None, None, None, 64, 64, 0, 2, None, None, None, 0, None) == 1


def test_product_refuses_rows_and_units_beyond_its_numbers(lib):
    import torch
    L = lib.lib()
    cfg = lib.config(2, 4, 64, 2, 4, torch.bfloat16)
    aligned = 1 << 20  # no call gets as far as to use these
    call = lambda n, k: L.moe_expert_product(ctypes.byref(cfg), aligned, aligned, aligned, aligned, aligned, n, k, 0, 2,  # noqa: E731
                                             aligned, None, aligned, 0, None)
    assert call(64, 1 << 30) == call(64, 64) == 3  # the workspace's size is refused, and nothing before it
    assert call(64, (1 << 30) + 32) == 1 and call(64, (1 << 31) - 32) == 1
    assert call(1 << 29, 64) == 1
    cfg.bs = 1 << 20  # 65540 row tiles at most: a CTA's next unit has to fit 32 bits too
    assert call(32766 * 64, 64) == 1 and call(32764 * 64, 64) == 3


def test_binding_refuses_cpu_tensors(lib):
    import torch
    rc = lib.router_config(4, 64, 8, torch.float32)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        lib.route(rc, x, None, torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8))
    with pytest.raises(ValueError):
        lib.mx_quantize(x, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))


def test_binding_refuses_other_configurations(lib):
    import torch
    x, ids, w = torch.zeros(4, 64), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    with pytest.raises(ValueError):
        lib.route(lib.config(2, 4, 64, 2, 4, torch.bfloat16), x, None, ids, w)
    with pytest.raises(TypeError):
        lib.route(None, x, None, ids, w)
    with pytest.raises(ValueError):
        lib.expert_product(lib.router_config(4, 64, 8, torch.float32), x, x, ids, x, x, x, ws=x)


def test_plain_quantiser_rounds_to_nearest_even():
    m = np.array([0.0, 0.25, 0.2501, 0.75, 0.7499, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 7.9])
    assert P.nearest_code(m).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 7]
