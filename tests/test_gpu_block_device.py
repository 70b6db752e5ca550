"""What a layer holds on another device than its input is refused before anything
is enqueued. (Weights on the host stand for another device here.)"""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import block as b

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M", [2, 20, 100])
def test_linear_refuses_weights_elsewhere(M):
    layer = g.Mx4Linear.from_weight(torch.ones(64, 96, device=DEV), backward=True)
    x, dy = torch.ones(M, 96, device=DEV), torch.ones(M, 64, device=DEV)
    w, wt = layer.weight, layer.weight_t
    for bad in (b._mx4(w.codes.cpu(), w.scales, w.k), b._mx4(w.codes, w.scales.cpu(), w.k)):
        layer.weight = bad
        with pytest.raises(ValueError, match="the weight's (codes|scales) must be a device tensor"):
            layer.forward(x)
    layer.weight = w
    for bad in (b._mx4(wt.codes.cpu(), wt.scales, wt.k), b._mx4(wt.codes, wt.scales.cpu(), wt.k)):
        layer.weight_t = bad
        with pytest.raises(ValueError, match="weight_t's (codes|scales) must be a device tensor"):
            layer.backward(dy, x)
        dx, dw = layer.backward(dy, x, need_dx=False)   # does not read it
        assert dx is None and dw.shape == (64, 96)
    layer.weight_t = wt
    assert bool((layer.forward(x) == 96).all()) and bool((layer.backward(dy, x)[0] == 64).all())


def test_layers_refuse_mixed_devices_at_construction():
    q = g.mx4_quantize(torch.ones(64, 96, device=DEV))
    for bad in (g.Mx4(q.codes, q.scales.cpu(), q.k), g.Mx4(q.codes.cpu(), q.scales, q.k)):
        with pytest.raises(ValueError, match="on the device"):
            g.Mx4Linear(bad)


def test_moe_refuses_a_layer_elsewhere():
    E, H, I = 3, 64, 32
    up, down = torch.ones(E, 2 * I, H, device=DEV).bfloat16(), torch.ones(E, H, I, device=DEV).bfloat16()
    layer = g.MoeLayer(torch.ones(E, H, device=DEV).bfloat16(), up, down, top_k=2)
    x = torch.ones(2, H, device=DEV).bfloat16()
    want = layer(x)
    keep, layer._keep = layer._keep, tuple(t.cpu() for t in layer._keep)
    with pytest.raises(ValueError, match="the layer must be a device tensor"):
        layer(x)
    layer._keep = keep
    assert torch.equal(layer(x), want)
