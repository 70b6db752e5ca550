"""Launch variants that larger layers take: the down product's 32-column blocks
over several groups of experts, the wide MXFP4 up product with many tokens on an
expert, and the few-rows MXFP4 product with two blocks of W and with runs of K
that reload the scales."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref
import test_gpu_block_moe as tm
import test_gpu_block_mx4 as tx

pytestmark = pytest.mark.gpu


# H / 32 * groups >= 256 and more than one group; H that ends inside a block of 32 columns
@pytest.mark.parametrize("kind", ["bf16", "f16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k", [(12, 4096, 24, 16, 4), (40, 4096, 40, 20, 3), (9, 4120, 16, 17, 2), (64, 2768, 8, 24, 6),
                                       (25, 4109, 13, 12, 8)])
def test_down_of_32_columns_and_several_groups(T, H, I, E, k, kind):
    assert H // 32 * -(-min(T * k, E) // 8) >= 256 and min(T * k, E) > 8
    tm.run(T, H, I, E, k, kind, renorm=E % 2 == 0, seed=T + H)


# ceil(I / 8) * 8 / 32 * min(T k, E) >= 512: 32 rows of each matrix a wave; 9 to 16, 17 to 32 and more tokens an expert
@pytest.mark.parametrize("T,H,I,E,k", [(8, 72, 8192, 2, 2), (13, 72, 8200, 2, 2), (16, 136, 4096, 4, 4), (30, 72, 8192, 2, 2),
                                       (64, 40, 5480, 3, 3), (41, 264, 4104, 4, 4)])
def test_wide_up_of_mxfp4(T, H, I, E, k):
    assert (I + 7) // 8 * 8 // 32 * min(T * k, E) >= 512
    tm.run(T, H, I, E, k, "mx4", renorm=T % 2 == 0, seed=T + I)


def few(M, N, K, dtype, seed):
    """run_linear with W drawn on the device: large ones take the host's packing too long."""
    x = tx.draw(M, K, dtype, seed)
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    w = (0.05 * torch.randn(N, K, generator=gen, device="cuda:0")).bfloat16()
    q = g.mx4_quantize(w)
    layer = g.Mx4Linear(q)
    print(f"[gpu] few rows M={M} N={N} K={K} {dtype}", flush=True)
    y = layer.forward(x.to("cuda:0"))
    # the codes' values, which the quantiser's tests hold to the definition, and x by the definition; in 64 bits
    wv = g.mx4_dequantize(q).double()
    r, e = ref.matmul_bound(ref.quantize(x)[0].to("cuda:0"), wv, 2.0 ** -8)
    ref.check(y, r.cpu(), e.cpu(), "y")
    layer.close()


@pytest.mark.parametrize("M", [1, 2, 7, 16, 24, 33, 64])
@pytest.mark.parametrize("N,K", [(4100, 520), (8192, 256), (8200, 1029), (12288, 300), (28672, 264)])
def test_few_rows_of_many_columns(M, N, K):
    few(M, N, K, "bf16" if M % 2 else "f16", M + N)


@pytest.mark.parametrize("M", [1, 4, 8, 9, 20, 40])
@pytest.mark.parametrize("N,K", [(24, 8192), (40, 8200), (40, 8449), (17, 20000), (8200, 8704)])
def test_few_rows_of_long_rows(M, N, K):
    few(M, N, K, "f32" if M == 4 else "bf16", M + K)
