"""The layers' weights in other layouts than contiguous ones, as a checkpoint of transposed matrices has them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from combine_route_scan_gb300 import build as B
    from combine_route_scan_gb300 import moe as M
    from combine_route_scan_gb300.int8_layer import Int8Layer
    from combine_route_scan_gb300.mxfp4_layer import Mxfp4Layer
    from test_int8_layer_gpu import make
    B.build()


def transposed(w):
    return w.transpose(1, 2).contiguous().transpose(1, 2)


def slices(w):
    return torch.cat((w, w), -1)[..., : w.shape[-1]]


@pytest.mark.parametrize("view", [transposed, slices])
@pytest.mark.parametrize("which", ["int8", "mxfp4"])
def test_weights_that_are_views(which, view):
    kind = Int8Layer if which == "int8" else Mxfp4Layer
    layer, x, logits, weights = make(kind=kind)
    views = [view(w) for w in weights]
    assert not any(v.is_contiguous() for v in views) and all(torch.equal(v, w) for v, w in zip(views, weights))
    other = kind(x.shape[0], x.shape[1], layer.ids.shape[-1], *views)
    assert torch.equal(layer(x, logits), other(x, logits))
    assert M.get_device_status(layer.ws) == 0 and M.get_device_status(other.ws) == 0
