"""Layers that are dropped while a call of theirs waits on another stream."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WAIT = 20_000_000   # clock ticks that the other stream is held up: some 10 ms


def overwrite(shapes):
    """Tensors of these shapes, where memory that was given back would go, full of NaN."""
    return [torch.full(s, 255, dtype=torch.uint8, device=DEV) for s in shapes for _ in range(3)]


@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_dropped_after_its_call(M):
    s = torch.cuda.Stream()
    w, x = torch.randn(1024, 2048, device=DEV).bfloat16(), torch.randn(M, 2048, device=DEV).bfloat16()
    dy = torch.randn(M, 1024, device=DEV).bfloat16()
    held = g.Mx4Linear.from_weight(w, backward=True)
    want = [held.forward(x), *held.backward(dy, x)]
    for _ in range(3):
        layer = g.Mx4Linear.from_weight(w, backward=True)
        shapes = [t.shape for q in (layer.weight, layer.weight_t) for t in (q.codes, q.scales)]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
        got = [layer.forward(x, stream=s), *layer.backward(dy, x, stream=s)]
        del layer
        kept = overwrite(shapes)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del kept


@pytest.mark.parametrize("packed", [False, True])
def test_moe_dropped_after_its_call(packed):
    s = torch.cuda.Stream()
    E, H, I = 4, 512, 256
    router, x = torch.randn(E, H, device=DEV).bfloat16(), torch.randn(5, H, device=DEV).bfloat16()

    def weights():
        gen = torch.Generator(device=DEV).manual_seed(3)
        up, down = (torch.randn(*n, generator=gen, device=DEV).bfloat16() / 16 for n in ((E, 2 * I, H), (E, H, I)))
        if not packed:
            return up, down
        qs = [g.mx4_quantize(w.reshape(-1, w.shape[-1])) for w in (up, down)]
        return [g.Mx4(q.codes.view(E, -1, q.codes.shape[1]), q.scales.view(E, -1, q.scales.shape[1]), q.k) for q in qs]

    want = g.MoeLayer(router, *weights(), top_k=2)(x)
    for _ in range(3):
        layer = g.MoeLayer(router.clone(), *weights(), top_k=2)
        shapes = [(t.numel() * t.element_size(),) for w in layer._keep
                  for t in ((w.codes, w.scales) if isinstance(w, g.Mx4) else (w,))]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
        got = layer(x, stream=s)
        del layer
        kept = overwrite(shapes)
        s.synchronize()
        assert torch.equal(got, want)
        del kept
