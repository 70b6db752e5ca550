"""The MXFP4 linear layer's tile path on values that are none, and both passes on
sizes of zero."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref
import test_gpu_block_mx4 as tx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M,N,K", [(100, 70, 300), (300, 512, 2304), (512, 256, 512)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_tile_path_keeps_nan_to_its_row_and_column(M, N, K, value):
    x, w = tx.draw(M, K, "bf16", 1), tx.draw(N, K, "bf16", 2)
    x[3, 5] = value
    x[M - 1, K - 1] = value
    q = g.mx4_quantize(w.to(DEV), 1)
    q.scales[7, 2] = 255
    y = g.Mx4Linear(q).forward(x.to(DEV)).cpu()
    nan = torch.zeros(M, N, dtype=torch.bool)
    nan[3], nan[M - 1], nan[:, 7] = True, True, True
    assert torch.equal(torch.isnan(y), nan)


def test_backward_keeps_nan_to_its_rows():
    M, N, K = 130, 96, 200
    dy, x, w = tx.draw(M, N, "bf16", 1), tx.draw(M, K, "bf16", 2), tx.draw(N, K, "bf16", 3, 0, 0.1)
    dy[9, 4] = float("nan")
    x[70, 11] = float("inf")
    dx, dw = g.Mx4Linear.from_weight(w.to(DEV), backward=True).backward(dy.to(DEV), x.to(DEV))
    bad_x, bad_w = torch.zeros(M, K, dtype=torch.bool), torch.zeros(N, K, dtype=torch.bool)
    bad_x[9] = True
    bad_w[4], bad_w[:, 11] = True, True
    assert torch.equal(torch.isnan(dx).cpu(), bad_x) and torch.equal(torch.isnan(dw).cpu(), bad_w)


@pytest.mark.parametrize("M,N,K", [(5, 0, 64), (100, 0, 64), (5, 32, 0), (100, 32, 0), (0, 32, 64)])
def test_sizes_of_zero(M, N, K):
    w = torch.ones(N, K, device=DEV).bfloat16()
    layer = g.Mx4Linear.from_weight(w, backward=True)
    x, dy = torch.ones(M, K, device=DEV).bfloat16(), torch.ones(M, N, device=DEV).bfloat16()
    y = layer.forward(x)
    dx, dw = layer.backward(dy, x)
    assert y.shape == (M, N) and dx.shape == (M, K) and dw.shape == (N, K)
    assert not bool(y.any()) and not bool(dx.any()) and not bool(dw.any())
    layer.close()


@pytest.mark.parametrize("shape", [(0, 64), (64, 0), (0, 0)])
def test_quantiser_on_nothing(shape):
    a, b = g.mx4_quantize(torch.empty(*shape, device=DEV), "both")
    assert a.rows == shape[0] and b.rows == shape[1]
    assert g.mx4_dequantize(a).shape == shape and g.mx4_dequantize(b).shape == shape[::-1]
    assert ref.padded(shape[1]) // 2 == a.codes.shape[1]
