"""The bits and the range of h between the mixture-of-experts layer's products.

Most cases here are exact: the gate is a power of two past which exp(-g) is
nothing to 1, so silu(g) = g, and every product and sum fits fp32. Then a
difference of two h shows whatever h lost on its way to the down product."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref
import test_gpu_block_moe as tm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def differences(dtype, T, E, k, gate, unit, down, H=96, I=72):
    """Layer whose h[0] = gate unit (1 + 2^-12 + 2^-20) and h[1] = gate unit (1 + 2^-12)
    in every expert, and whose out[n] is down (h[0] - h[1]) in every third column, else 0."""
    x = torch.zeros(T, H, dtype=dtype)
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = gate[0], unit[0], unit[0] * 2.0 ** -6, unit[0] * 2.0 ** -10
    up, dn = torch.zeros(E, 2 * I, H), torch.zeros(E, H, I)
    up[:, :2, 0] = gate[1]
    up[:, I:I + 2, 1], up[:, I:I + 2, 2] = unit[1], unit[1] * 2.0 ** -6
    up[:, I, 3] = unit[1] * 2.0 ** -10
    dn[:, ::3, 0], dn[:, ::3, 1] = down, -down
    assert torch.equal(up.to(dtype).double(), up.double()) and torch.equal(dn.to(dtype).double(), dn.double())
    router = torch.zeros(E, H, dtype=dtype)   # every expert alike: the lowest indices, each with a share of 1 / k
    want = torch.zeros(T, H)
    want[:, ::3] = gate[0] * gate[1] * unit[0] * unit[1] * 2.0 ** -20 * down
    return x, router, up.to(dtype), dn.to(dtype), want


def exact(dtype, T, E, k, **kw):
    x, router, up, dn, want = differences(dtype, T, E, k, **kw)
    assert torch.equal(want.to(dtype).float(), want) and bool(want.any())
    layer = g.MoeLayer(router.to(DEV), up.to(DEV), dn.to(DEV), top_k=k)
    print(f"[gpu] moe h {dtype} T={T} E={E} k={k} {kw}", flush=True)
    got = layer(x.to(DEV)).cpu().float()
    assert torch.equal(got, want), f"off by {float((got - want).abs().max())} of {float(want.max())}"


# tokens on each expert: 1, 5 and 6 to 8 (fewer and more than one tile of columns takes), 9 to 16, more
COUNTS = [(1, 2, 1), (5, 1, 1), (6, 1, 1), (8, 2, 2), (9, 1, 1), (16, 2, 2), (17, 1, 1), (64, 2, 2), (3, 32, 16)]


@pytest.mark.parametrize("T,E,k", COUNTS)
def test_bf16_h_keeps_24_bits(T, E, k):
    exact(torch.bfloat16, T, E, k, gate=(16.0, 8.0), unit=(1.0, 1.0), down=1.0)


@pytest.mark.parametrize("T,E,k", COUNTS)
def test_fp16_h_keeps_22_bits(T, E, k):
    exact(torch.float16, T, E, k, gate=(16.0, 8.0), unit=(1.0, 1.0), down=2.0 ** 4)
    # h of 2^-8, whose second number would be below fp16's steps were it not scaled
    exact(torch.float16, T, E, k, gate=(16.0, 8.0), unit=(2.0 ** -7, 2.0 ** -8), down=2.0 ** 14)


@pytest.mark.parametrize("T,E,k", COUNTS)
def test_fp16_h_beyond_fp16(T, E, k):
    """h of 2^20 and of 2^50, which fp16 does not hold, in a layer whose output it does."""
    exact(torch.float16, T, E, k, gate=(2.0 ** 5, 2.0 ** 5), unit=(2.0 ** 5, 2.0 ** 5), down=2.0 ** -10)
    exact(torch.float16, T, E, k, gate=(2.0 ** 13, 2.0 ** 12), unit=(2.0 ** 13, 2.0 ** 12), down=2.0 ** -20)


@pytest.mark.parametrize("T,H,I,E,k", [(5, 64, 40, 4, 2), (40, 264, 72, 6, 2), (64, 2056, 24, 17, 3), (33, 4104, 16, 12, 4)])
def test_fp16_large_h_of_some_tokens(T, H, I, E, k):
    """Tokens of all magnitudes, h up to 10^7, against the 64-bit form."""
    x, router, up, down, up64, down64 = tm.make(T, H, I, E, "f16", T + H)
    x = (x.float() * torch.logspace(-2, 1.5, T).unsqueeze(1)).half()
    router = (router.float() * 0.03).half()
    up64 = (up64 * 20).half().double()
    down64 = (down64 * 2.0 ** -7).half().double()
    layer = g.MoeLayer(router.to(DEV), up64.half().to(DEV), down64.half().to(DEV), top_k=k)
    out, ids, _ = layer(x.to(DEV), return_routing=True)
    rids, rp = ref.route(x, router, k, True)
    assert torch.equal(ids.cpu().long(), rids)
    gu = x.double() @ up64[rids[-1, 0]].t()
    assert float((gu[-1, :I] * gu[-1, I:]).abs().max()) > 65504
    r, e = ref.moe(x, up64, down64, rids, rp, ref.HALF[torch.float16])
    ref.check(out, r, e, "out")
    assert torch.equal(layer(x.to(DEV)), out), "not the same bits twice"


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinite_h_spoils_its_token_alone(kind):
    x, router, up, down, up64, down64 = tm.make(9, 200, 72, 6, kind, 7)
    x[4, 11] = float("inf")
    out = g.MoeLayer(router.to(DEV), up, down, top_k=2)(x.to(DEV)).cpu()
    assert not bool(torch.isfinite(out[4]).any())
    rest = [i for i in range(9) if i != 4]
    rids, rp = ref.route(x[rest], router, 2, True)
    r, e = ref.moe(x[rest], up64, down64, rids, rp, ref.HALF[x.dtype])
    ref.check(out[rest], r, e, "out")


@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (6, 1, 1), (64, 2, 2)])
def test_mxfp4_h_keeps_24_bits(T, E, k):
    """The same differences with MXFP4 weights (powers of two are exact in them)."""
    x, router, up, dn, want = differences(torch.bfloat16, T, E, k, gate=(16.0, 8.0), unit=(1.0, 1.0), down=1.0,
                                          H=128, I=72)
    # an expert's rows of 32 share a scale: 2^-6 and 2^-10 beside 1 go to blocks of their own
    x4, up4 = torch.zeros_like(x), torch.zeros_like(up)
    for i in range(4):
        x4[:, 32 * i], up4[:, :, 32 * i] = x[:, i], up[:, :, i]
    parts = []
    for w in (up4, dn):
        c, s, v = zip(*(ref.pack(m) for m in w))
        assert torch.equal(torch.stack(v), w.double())
        parts.append(g.Mx4(torch.stack(c).to(DEV), torch.stack(s).to(DEV), w.shape[2]))
    out = g.MoeLayer(torch.zeros(E, 128, dtype=torch.bfloat16, device=DEV), *parts, top_k=k)(x4.to(DEV))
    want = torch.zeros(T, 128)
    want[:, ::3] = 128.0 * 2.0 ** -20
    assert torch.equal(out.cpu().float(), want), f"off by {float((out.cpu().float() - want).abs().max())}"
