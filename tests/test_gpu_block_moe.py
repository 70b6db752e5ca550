"""The mixture-of-experts layer against the 64-bit form of block_ref."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, I, E, kind, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    rnd = lambda *s, std: (torch.randn(*s, generator=gen) * std).to(dt)  # noqa: E731
    x = rnd(T, H + pad, std=1.0)[:, :H]
    router = rnd(E, H, std=2 / H ** 0.5)
    up, down = rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=max(I, 1) ** -0.5)
    if kind != "mx4":
        return x, router, up.to(DEV), down.to(DEV), up.double(), down.double()
    packed, values = [], []
    for w in (up, down):
        c, s, v = zip(*(ref.pack(m) for m in w))
        packed.append(g.Mx4(torch.stack(c).to(DEV), torch.stack(s).to(DEV), w.shape[2]))
        values.append(torch.stack(v))
    return x, router, *packed, *values


def run(T, H, I, E, k, kind, renorm=True, pad=0, mask=None, seed=0):
    x, router, up, down, up64, down64 = make(T, H, I, E, kind, seed, pad)
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=k, renormalize=renorm)
    xd = torch.full((T, H + pad), float("nan"), dtype=x.dtype, device=DEV)
    xd[:, :H] = x.to(DEV)
    if mask is not None:
        xd[~mask.to(DEV)] = float("nan")   # masked tokens hold anything
    guard = torch.full((T + 2, H), 77.0, dtype=x.dtype, device=DEV)
    print(f"[gpu] moe T={T} H={H} I={I} E={E} k={k} {kind} renorm={renorm} pad={pad} masked={mask is not None}",
          flush=True)
    out, ids, p = layer(xd[:, :H], mask.to(DEV) if mask is not None else None, return_routing=True, out=guard[1:-1])
    torch.cuda.synchronize()
    assert bool((guard[0] == 77).all()) and bool((guard[-1] == 77).all()), "wrote outside out"
    rids, rp = ref.route(x, router, k, renorm, mask)
    assert torch.equal(ids.cpu().long(), rids)
    ref.check(p, rp, 2.0 ** -23 * rp + 1e-37, "probs")
    r, e = ref.moe(x, up64, down64, rids, rp, ref.HALF[x.dtype])
    ref.check(out, r, e, "out")
    again = layer(xd[:, :H], mask.to(DEV) if mask is not None else None)
    assert torch.equal(again, out), "not the same bits twice"
    return layer


@pytest.mark.parametrize("kind", ["bf16", "f16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (3, 264, 72, 5, 5), (16, 128, 96, 4, 1), (17, 512, 40, 16, 4),
                                       (64, 192, 64, 3, 2), (40, 320, 16, 70, 8), (64, 128, 32, 100, 16)])
def test_layer(T, H, I, E, k, kind):
    run(T, H, I, E, k, kind, renorm=T % 2 == 1, seed=T + H)


@pytest.mark.parametrize("kind", ["bf16", "f16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k,pad", [(1, 1, 1, 1, 1, 0), (5, 33, 17, 6, 2, 1), (9, 257, 259, 4, 3, 0), (18, 130, 67, 2, 1, 5)])
def test_odd_sizes(T, H, I, E, k, pad, kind):
    run(T, H, I, E, k, kind, renorm=False, pad=pad, seed=H)


@pytest.mark.parametrize("kind", ["bf16", "f16", "mx4"])
@pytest.mark.parametrize("E,k", [(16, 16), (64, 9), (65, 8), (130, 16), (512, 7)])
def test_one_token_on_many_experts(E, k, kind):
    run(1, 136, 24, E, k, kind, renorm=k % 2 == 0, seed=E)


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 9100, 40, 3, 2), (2, 48, 4500, 3, 2), (5, 40, 4612, 10, 3), (20, 8452, 16, 2, 1)])
def test_long_rows(T, H, I, E, k, kind):
    run(T, H, I, E, k, kind, seed=H)


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("T,keep", [(1, []), (6, []), (6, [2]), (33, [0, 5, 6, 7, 32])])
def test_masked_tokens(T, keep, kind):
    mask = torch.zeros(T, dtype=torch.bool)
    mask[keep] = True
    run(T, 160, 48, 8, 2, kind, mask=mask, seed=T)


def test_all_tokens_on_one_expert_and_most_experts():
    run(64, 64, 32, 1, 1, "bf16")
    run(2, 64, 32, 512, 16, "bf16")


def test_ties_take_the_lowest_index():
    """Whole-number logits are exact, so equal ones are ties."""
    H, E, k = 64, 40, 6
    gen = torch.Generator().manual_seed(4)
    x = torch.randint(-2, 3, (20, H), generator=gen).bfloat16()
    router = torch.randint(-1, 2, (4, H), generator=gen).bfloat16().repeat(10, 1)   # every logit ten times
    up, down = torch.zeros(E, 16, H, device=DEV).bfloat16(), torch.zeros(E, H, 8, device=DEV).bfloat16()
    for renorm in (True, False):
        layer = g.MoeLayer(router.to(DEV), up, down, top_k=k, renormalize=renorm)
        _, ids, p = layer(x.to(DEV), return_routing=True)
        rids, rp = ref.route(x, router, k, renorm)
        assert torch.equal(ids.cpu().long(), rids)
        ref.check(p, rp, 2.0 ** -23 * rp, "probs")


def test_nan_stays_with_its_token():
    x, router, up, down, up64, down64 = make(6, 128, 32, 8, "bf16", 1)
    x[2, 7] = float("nan")
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=2)
    out, ids, p = layer(x.to(DEV), return_routing=True)
    rids, rp = ref.route(x, router, 2, True)
    assert torch.equal(ids.cpu().long(), rids)
    assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(p[2]).all())
    rest = [0, 1, 3, 4, 5]
    r, e = ref.moe(x[rest], up64, down64, rids[rest], rp[rest], ref.HALF[x.dtype])
    ref.check(out[rest], r, e, "out")


def test_one_nan_expert_comes_last():
    """A router row of NaN makes that logit NaN for every token: it is chosen
    only where nothing else is left."""
    x, router, up, down, *_ = make(3, 64, 16, 4, "bf16", 2)
    router[1] = float("nan")
    out, ids, p = g.MoeLayer(router.to(DEV), up, down, top_k=3)(x.to(DEV), return_routing=True)
    assert not bool((ids == 1).any()) and bool(torch.isfinite(out).all())
    _, ids, p = g.MoeLayer(router.to(DEV), up, down, top_k=4)(x.to(DEV), return_routing=True)
    assert bool((ids[:, 3] == 1).all()) and bool(torch.isnan(p).all())


def test_empty_and_inner_zero():
    x, router, up, down, *_ = make(4, 64, 16, 4, "bf16", 2)
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=2)
    assert layer(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)).shape == (0, 64)
    none = g.MoeLayer(router.to(DEV), up[:, :0].contiguous(), down[:, :, :0].contiguous(), top_k=2)
    assert not bool(none(x.to(DEV)).any())


def test_two_streams():
    """Each stream has counters of its own."""
    x, router, up, down, *_ = make(32, 512, 256, 16, "bf16", 3)
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=4)
    xd = x.to(DEV)
    want = layer(xd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got.append(layer(xd, stream=s))
        got.append(layer(xd))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


def test_graph_replays():
    x, router, up, down, *_ = make(8, 256, 64, 16, "mx4", 3)
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=4)
    xd = x.to(DEV)
    layer(xd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(xd)
    for i in range(4):
        xd.copy_(x.roll(i, 0))
        want = layer(xd).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
