"""Without a device: the plan's device is asked for before the linear layer
enqueues anything, at every number of rows. (Where there is a device these calls
would run on addresses that are none.)"""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import block as b   # noqa: F401  (declares the C entries)

P = 1 << 20
BF16 = int(g.Dtype.BF16)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")
@pytest.mark.parametrize("M", [1, 8, 9, 64, 65])
def test_linear_asks_for_the_plans_device_first(M):
    plan = g.Plan("f4e2m1", la="row", lb="col", lc="row")
    status = g.lib.gemm_mx4_linear(plan.handle, P, BF16, 64, P, P, None, P, M, 8, 64, P, 1 << 30, None)
    assert status == g.Status.HIP_ERROR and "hipGetDevice" in g.lib.gemm_last_error().decode()
    status = g.lib.gemm_mx4_linear_backward(plan.handle, P, 8, P, 64, BF16, P, P, P, P, M, 8, 64, P, 1 << 30, None)
    assert status == g.Status.HIP_ERROR and "hipGetDevice" in g.lib.gemm_last_error().decode()
    plan.close()
