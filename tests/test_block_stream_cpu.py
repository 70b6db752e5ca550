"""A layer called with ``stream`` keeps its own tensors, not its arguments'
alone, from reuse until that stream has passed the call: the layer may be
dropped right after it. Shown on stand-ins for device tensors that note the
streams they are recorded on; the calls end at the binding's checks."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import block as b


class Device(torch.Tensor):
    """A host tensor that says it is on the device."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        noted.append((id(self), stream))


noted = []


def tensor(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


def linear():
    layer = object.__new__(g.Mx4Linear)
    layer.weight, layer.weight_t = (b._mx4(tensor(8, 128), tensor(8, 8), 64) for _ in range(2))
    layer.N = layer.K = 64
    layer.plan = g.Plan("f4e2m1", la="row", lb="col", lc="row")
    return layer


def recorded(call, stream):
    noted.clear()
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        call()
    assert all(s is stream for _, s in noted)
    return {i for i, _ in noted}


def test_linear_keeps_its_weights():
    layer, s, x = linear(), object(), tensor(4, 64, dtype=torch.float32)
    assert {id(layer.weight.codes), id(layer.weight.scales), id(x)} <= recorded(lambda: layer.forward(x, stream=s), s)
    assert {id(layer.weight_t.codes), id(layer.weight_t.scales), id(x)} <= recorded(
        lambda: layer.backward(x, x, stream=s), s)
    layer.weight_t = None   # the gradient of W alone reads no weight
    assert id(x) in recorded(lambda: layer.backward(x, x, need_dx=False, stream=s), s)
    layer.close()


@pytest.mark.parametrize("packed", [False, True])
def test_moe_keeps_its_weights(packed):
    layer, s, x = object.__new__(g.MoeLayer), object(), torch.zeros(2, 64, dtype=torch.bfloat16)
    router = tensor(4, 64)
    up, down = ((b._mx4(tensor(4, 8, 128), tensor(4, 8, 8), 64) if packed else tensor(4, 8, 64)) for _ in range(2))
    layer._keep, layer._at = (router, up, down), None   # x is a host tensor: refused before the call
    own = {id(router)} | {id(t) for w in (up, down) for t in ((w.codes, w.scales) if packed else (w,))}
    assert own <= recorded(lambda: layer(x, stream=s), s)
