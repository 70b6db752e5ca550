"""The operators together, and calls at the borders of their variants: more
tokens on one expert than a tile holds, experts beyond one group, sums that
end inside a chunk, rows that workgroups walk over, the longest rows, tensors
of other streams, captured calls."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import feed_forward as ff
import block_ref as ref
import test_gpu_block_moe as tm
import test_gpu_block_mx4 as tx
import test_gpu_block_norm as tn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["bf16", "f16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k", [
    (64, 72, 40, 2, 2),        # 64 tokens on each expert, one group whose waves share K
    (50, 136, 264, 1, 1),      # one expert
    (33, 264, 136, 9, 9),      # two groups, 33 tokens on each expert
    (64, 520, 24, 17, 3),      # three groups, the last of one expert
    (5, 1032, 520, 128, 4),    # 128 experts
    (7, 40, 200, 129, 16),     # over 128 experts, the most choices
    (64, 64, 16, 512, 16),     # the most experts and slots
    (2, 2056, 2304, 4, 2),     # MXFP4 runs of more units than one load of scales covers
])
def test_moe_borders(T, H, I, E, k, kind):
    tm.run(T, H, I, E, k, kind, renorm=E % 2 == 0, seed=T + E)


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("H,I", [(65, 63), (127, 129), (1025, 1001), (4, 7)])
def test_moe_sums_that_end_inside_a_chunk(H, I, kind):
    tm.run(20, H, I, 12, 3, kind, seed=H)


def test_moe_masked_groups():
    """Masked tokens leave whole groups without experts; the others' bits stay."""
    T = 40
    x, router, up, down, *_ = tm.make(T, 256, 64, 64, "bf16", 5)
    layer = g.MoeLayer(router.to(DEV), up, down, top_k=6)
    xd = x.to(DEV)
    want = layer(xd)
    for keep in ([], [3], [0, 39], list(range(0, 40, 2))):
        mask = torch.zeros(T, dtype=torch.bool, device=DEV)
        mask[keep] = True
        got = layer(xd, mask)
        assert torch.equal(got[mask], want[mask]) and not bool(got[~mask].any())


def test_moe_infinite_token():
    """An infinity spoils its own token alone."""
    x, router, up, down, up64, down64 = tm.make(9, 200, 72, 6, "bf16", 7)
    x[4, 11] = float("inf")
    out = g.MoeLayer(router.to(DEV), up, down, top_k=2)(x.to(DEV)).cpu()
    assert not bool(torch.isfinite(out[4]).any())
    rest = [i for i in range(9) if i != 4]
    rids, rp = ref.route(x[rest], router, 2, True)
    r, e = ref.moe(x[rest], up64, down64, rids, rp, ref.HALF[x.dtype])
    ref.check(out[rest], r, e, "out")


def test_moe_carries_more_than_the_type():
    """h in two numbers: the result is within the bound that a rounded h would
    need for its output's rounding and the sums alone."""
    x, router, up, down, up64, down64 = tm.make(6, 512, 256, 4, "bf16", 9)
    out, ids, p = g.MoeLayer(router.to(DEV), up, down, top_k=2)(x.to(DEV), return_routing=True)
    rids, rp = ref.route(x, router, 2, True)
    # h off by 2^-16 instead of 2^-8, the output rounded to bf16
    r, e = ref.moe(x, up64, down64, rids, rp, 2.0 ** -16)
    ref.check(out, r, e + 2.0 ** -8 * r.abs(), "out")


@pytest.mark.parametrize("M,N,K", [(3, 8193, 264), (8, 40, 1300), (9, 8200, 1029), (40, 8192, 136), (47, 33, 2050),
                                   (64, 8208, 300), (65, 130, 513), (300, 1001, 520), (1, 16, 4100), (2, 5, 31)])
@pytest.mark.parametrize("act", ["linear", "relu"])
def test_linear_borders(M, N, K, act):
    tx.run_linear(M, N, K, "f32" if M % 3 == 0 else "bf16", M != 64, M % 4, M + K, act)


def test_linear_other_activations():
    """The GEMM's other epilogues keep to its element-wise path."""
    x, w = tx.draw(90, 100, "bf16", 1), tx.draw(70, 100, "bf16", 2, 0, 0.1)
    xv, wv = ref.quantize(x)[0], ref.quantize(w)[0]
    for act, fn in (("sigmoid", torch.sigmoid), ("tanh", torch.tanh)):
        y = g.Mx4Linear.from_weight(w.to(DEV), activation=act).forward(x.to(DEV))
        r, e = ref.matmul_bound(xv, wv, 0.0)
        # slope at most one; exp, division: 32 steps
        ref.check(y, fn(r), e + (2.0 ** -8 + 32 * ref.F32) * fn(r).abs() + 32 * ref.F32, act)


@pytest.mark.parametrize("T,H,dtype,groups", [(1100, 2048, "bf16", 0), (2100, 1000, "f32", 3), (1030, 4100, "bf16", 5),
                                              (300, 8192, "f32", 300), (20, 16384, "bf16", 4), (600, 9000, "bf16", 2),
                                              (300, 8201, "f32", 1), (4, 12000, "f16", 4)])
def test_norm_borders(T, H, dtype, groups):
    tn.run(tn.case(T, H, dtype, groups, pad=H % 3, seed=T))


@pytest.mark.parametrize("H", [1, 3, 7, 9, 15])
def test_norm_short_rows(H):
    for dtype in ("bf16", "f32"):
        tn.run(tn.case(9, H, dtype, 3, pad=2, seed=H), act="sigmoid")


def test_decoder_is_its_operators():
    d = ff.MoeDecoder(2, 256, 96, 8, 2, seed=3)
    x = torch.randn(5, 256, device=DEV).bfloat16()
    got = d(x)
    r, n = x, g.norm_residual(None, x, w_next=d.w_first)[1]
    for moe, w_post, scale, w_next in d.layers:
        y = moe(n)
        want, e = ref.norm_out(y.cpu(), r.cpu(), w_post.cpu(), None, scale.cpu(), 1e-6, "linear", 2.0 ** -8)
        r, n, _ = g.norm_residual(y, r, w_post=w_post, scale=scale, w_next=w_next)
        ref.check(r, want, e, "residual")
    assert torch.equal(got, n)


def test_decoder_graph_replays():
    d = ff.MoeDecoder(3, 512, 128, 16, 4, seed=1)
    x = torch.randn(8, 512, device=DEV).bfloat16()
    d(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d(x)
    for i in range(4):
        x.copy_(torch.randn(8, 512, device=DEV).bfloat16())
        want = d(x).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_training_step_learns():
    b = ff.DenseBlock(256, seed=2)
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(512, 256, generator=gen, device=DEV).bfloat16()
    target = torch.randn(512, 256, generator=gen, device=DEV).bfloat16()
    losses = [float(b.step(x, target, 100.0)) for _ in range(8)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_linear_graph_replays():
    """Forward (both kernels) and backward captured once the plan is warm."""
    w = torch.randn(192, 320, device=DEV).bfloat16()
    layer = g.Mx4Linear.from_weight(w, backward=True)
    for M in (4, 20, 200):
        x, dy = torch.randn(M, 320, device=DEV).bfloat16(), torch.randn(M, 192, device=DEV).bfloat16()

        def step():
            return [layer.forward(x), *layer.backward(dy, x)]

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for i in range(3):
            x.copy_(torch.randn(M, 320, device=DEV).bfloat16())
            want = [t.clone() for t in step()]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(held, want)), (M, i)


def test_stream_argument_keeps_its_tensors():
    """Inputs that die right after a call on another stream are not reused under it."""
    s = torch.cuda.Stream()
    w = torch.ones(2048, device=DEV, dtype=torch.bfloat16)
    for i in range(20):
        x = torch.full((2000, 2048), float(i + 1), device=DEV, dtype=torch.bfloat16)
        s.wait_stream(torch.cuda.current_stream())
        out = g.norm_residual(None, x, w_next=w, stream=s)[1]
        del x
        torch.full((2000, 2048), float("nan"), device=DEV, dtype=torch.bfloat16)
        s.synchronize()
        assert bool((out == 1).all()), i


def test_command_runs(capsys):
    ff.main(["--tokens", "3", "--layers", "2", "--hidden", "256", "--inner", "64", "--experts", "8", "--top-k", "2",
             "--steps", "2", "--rows", "64"])
    out = capsys.readouterr().out
    assert "is the eager one: True" in out and "training loss:" in out
