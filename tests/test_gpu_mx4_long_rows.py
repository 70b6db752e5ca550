"""The few-rows MXFP4 product at the longest K it takes, where the codes of x
span up to 2^31 bytes: the last elements of every row count."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M,K", [(64, 1 << 25), (63, 1 << 26), (64, 1 << 26), (64, (1 << 26) - 255), (1, 1 << 26)])
def test_last_elements_of_every_row(M, K):
    N = 3
    print(f"[gpu] mx4 long rows M={M} K={K}", flush=True)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(N, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0], w[:, 0] = 4.0, 1.0
    x[:, -3:] = torch.arange(M, device=DEV).remainder(4).add(1).unsqueeze(1)   # 1, 2, 3 or 4: exact in MXFP4
    w[:, -3:] = torch.arange(1, N + 1, device=DEV).unsqueeze(1)
    layer = g.Mx4Linear.from_weight(w)
    y = layer.forward(x).cpu().float()
    a, b = torch.arange(M).remainder(4).add(1).float(), torch.arange(1, N + 1).float()
    want = 4.0 + 3.0 * a[:, None] * b[None, :]
    layer.close()
    del x, w, layer
    torch.cuda.empty_cache()
    assert torch.equal(y, want), (y - want).abs().max(1).values.nonzero().flatten().tolist()
