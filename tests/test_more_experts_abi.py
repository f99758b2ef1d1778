"""The int8 operators and the gradients of combine and dispatch without a GPU: what
their entries refuse on the host, before they would touch a device."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
AT = 1 << 20  # an aligned address that no call gets as far as to use


@pytest.fixture(scope="module")
def lib():
    from combine_route_scan_gb300 import build
    build.build()
    from combine_route_scan_gb300 import moe
    return moe


@pytest.fixture
def cfg(lib):
    import torch
    return lib.config(2, 4, 64, 2, 4, torch.bfloat16)


def test_quantiser_refusals(lib):
    call = lambda dtype=2, mats=2, rows=3, cols=64, rs=64, ms=192, counts=None, n=0, x=AT, codes=AT, scales=AT: (  # noqa: E731
        lib.lib().moe_int8_quantize(x, dtype, mats, rows, cols, rs, ms, counts, n, codes, scales, None))
    for bad in (dict(dtype=0), dict(dtype=4), dict(mats=-1), dict(rows=-1), dict(cols=0), dict(cols=(1 << 30) + 1), dict(rs=63),
                dict(ms=-1), dict(rows=1 << 30), dict(rows=1 << 31, mats=1), dict(counts=AT, n=0), dict(counts=AT, n=4, mats=1025),
                dict(counts=AT + 2, n=4), dict(x=None), dict(codes=None), dict(scales=None), dict(x=AT + 1), dict(scales=AT + 2),
                dict(dtype=3, x=AT + 2)):
        assert call(**bad) == INVALID, bad
    assert call(mats=0) == 0 and call(rows=0) == 0  # nothing to do


def test_product_refusals(lib, cfg):
    call = lambda n=64, k=64, epi=0, yt=2, x=AT, xs=AT, ep=AT, w=AT, ws=AT, y=AT, space=AT, size=0: (  # noqa: E731
        lib.lib().moe_expert_product_int8(ctypes.byref(cfg), x, xs, ep, w, ws, n, k, epi, yt, y, space, size, None))
    assert call() == call(xs=None) == call(k=1) == call(k=131071) == WORKSPACE  # its size, and nothing before it
    for bad in (dict(n=0), dict(k=0), dict(k=131072), dict(epi=2), dict(epi=-1), dict(n=63, epi=1), dict(yt=0), dict(yt=3),
                dict(yt=4), dict(n=1 << 29), dict(x=None), dict(ep=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=AT + 8),
                dict(w=AT + 8), dict(y=AT + 8), dict(xs=AT + 2), dict(ep=AT + 2), dict(ws=AT + 1)):
        assert call(**bad) == INVALID, bad
    assert call(space=None) == WORKSPACE
    cfg.topk = 0
    assert call() == INVALID
    assert lib.lib().moe_expert_product_int8(None, AT, AT, AT, AT, AT, 64, 64, 0, 2, AT, AT, 0, None) == INVALID


NAMES = {"combine": ("grad_out", "expert_out", "assist", "ep", "ids", "scales", "mask", "x", "grad_rows", "grad_scales", "grad_x"),
         "dispatch": ("grad_rows", "assist", "ep", "ids", "mask", "residual", "grad_row_scales", "grad_x", "grad_scales")}


def backward(lib, which, cfg, space=AT, size=1 << 30, **arrays):
    entry = getattr(lib.lib(), f"moe_{which}_backward")
    return entry(ctypes.byref(cfg), *[arrays.get(a, AT) for a in NAMES[which]], space, size, None)


@pytest.mark.parametrize("which", ["combine", "dispatch"])
def test_backward_refusals(lib, cfg, which):
    import torch
    call = lambda **kw: backward(lib, which, cfg, **kw)  # noqa: E731
    assert call(size=0) == call(space=None) == call(space=AT + 16) == WORKSPACE
    for name in ("assist", "ep", "ids"):
        assert call(**{name: None}) == INVALID and call(**{name: AT + 2}) == INVALID, name
    aligned = {"combine": ("grad_out", "expert_out", "x", "grad_rows", "grad_x"), "dispatch": ("grad_rows", "residual", "grad_x")}
    for name in aligned[which]:
        assert call(**{name: AT + 8}) == INVALID, name
    assert call(grad_scales=AT + 2) == INVALID
    if which == "combine":
        assert call(grad_out=None) == INVALID and call(scales=None) == INVALID and call(scales=AT + 1) == INVALID
        assert call(expert_out=None) == INVALID  # the weights' gradient needs it
        assert call(grad_rows=None, grad_scales=None, grad_x=None) == INVALID
    else:
        assert call(grad_rows=None) == INVALID and call(grad_x=None) == INVALID
        assert call(grad_scales=None) == INVALID and call(grad_row_scales=None) == INVALID  # both or none
        assert call(grad_row_scales=AT + 2) == INVALID
    for kw in (dict(quant_mode=2), dict(quant_mode=4, expand_dtype="fp4_e2m1")):
        other = lib.config(2, 4, 64, 2, 4, torch.bfloat16, **kw)
        assert backward(lib, which, other) == UNSUPPORTED
    assert backward(lib, which, lib.config(2, 4, 64, 2, 4, torch.int32)) == UNSUPPORTED
    masked = lib.config(2, 4, 64, 2, 4, torch.bfloat16, mask_kind=2)
    assert backward(lib, which, masked, mask=None) == INVALID
    if which == "combine":
        copies = lib.config(2, 4, 64, 2, 4, torch.bfloat16, copy_expert_num=1)
        assert backward(lib, which, copies, x=None) == INVALID  # needed for the copies' weights
    empty = lib.config(2, 0, 64, 2, 4, torch.bfloat16)
    assert backward(lib, which, empty) == 0  # nothing to do
    cfg.bs = -1
    assert call() == INVALID


def test_binding_refuses_other_tensors_and_configurations(lib, cfg):
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.int8_quantize(x, x, x)
    with pytest.raises(ValueError):
        lib.expert_product_int8(cfg, x, None, x, x, x, x, ws=x)
    with pytest.raises(ValueError):
        lib.combine_backward(cfg, x, x, x, x, x, x, None, None, x, ws=x)
    with pytest.raises(ValueError):
        lib.dispatch_backward(lib.router_config(4, 64, 8, torch.float32), x, x, x, x, None, x, ws=x)
    with pytest.raises(TypeError):
        lib.dispatch_backward(None, x, x, x, x, None, x, ws=x)
