"""The MXFP4 product's epilogue with a scale and a bias: alpha times the sum is
rounded to fp32 before the bias is added, whichever path a tile takes."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def whole(rows, k, seed):
    """Whole numbers that MXFP4 holds, as (codes, scales, values)."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.randint(-3, 4, (rows, k), generator=gen).float()
    w[:, ::32] = 4.0
    c, s, v = ref.pack(w)
    assert torch.equal(v, w.double())
    return c.to(DEV), s.to(DEV), v


@pytest.mark.parametrize("act", [None, "relu"])
@pytest.mark.parametrize("M,N,K", [(512, 512, 512), (300, 520, 512), (333, 517, 256), (130, 1031, 2304), (1100, 1280, 512)])
def test_alpha_and_bias_round_apart(M, N, K, act):
    a, sa, av = whole(M, K, 1)
    b, sb, bv = whole(N, K, 2)
    acc = (av @ bv.t()).float()          # whole numbers below 2^24: exact in any order
    bias = (100 * torch.randn(N, generator=torch.Generator().manual_seed(3))).bfloat16()
    for alpha in (0.3, -0.7, 1.0):
        plan = g.Plan("f4e2m1", "bf16", "row", "col", "row", activation=act)
        d = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        print(f"[gpu] mx4 epilogue {M}x{N}x{K} alpha={alpha} {act}", flush=True)
        plan.run_mx(a, b, None, d, M, N, K, sa, sb, alpha, 0.0, bias=bias.to(DEV))
        want = acc * torch.tensor(alpha, dtype=torch.float32) + bias.float()
        if act:
            want = want.clamp_min(0)
        off = (d.cpu() != want.bfloat16()).sum()
        plan.close()
        assert int(off) == 0, f"{int(off)} of {M * N} values differ at alpha = {alpha}"
