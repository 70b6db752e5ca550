"""The losses of the output head and their gradients, against the 64-bit forms
of model_ref (computed on the device, in float64)."""
import math

import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import model_ref as ref
from block_ref import HALF

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def check(got, want, err, name):
    """|got - want| <= err; NaN in the same places. A type's largest value is
    (2 - eps) 2^e with steps of eps 2^e below it, so what rounds to infinity is
    from half a step above it on, eps / 4 of it: infinities are right where a
    value within err of want is that large, and wanted where all of them are."""
    t = torch.finfo(got.dtype)
    edge = t.max * (1 + t.eps / 4)
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    size, inf = want.abs(), torch.isinf(got)
    assert bool((inf | ~(size - err > edge * (1 + 1e-6))).all()), f"{name}: no infinity past the type's range"
    right = inf & (torch.sign(got) == torch.sign(want)) & (size + err >= edge * (1 - 1e-6))
    off = torch.where(torch.isnan(want) | right, 0.0, (got - want).abs() - err)
    assert not off.numel() or float(off.max()) <= 0, (
        f"{name}: {int((off > 0).sum())} of {off.numel()} outside, worst {float(off.max()):.3g} beyond a bound of "
        f"{float(err.flatten()[off.argmax()]):.3g}")


def rows(gen, n, c, dt, pad=0, std=1.0, shift=0):
    """N(0, std^2) rows on the device with NaN between them."""
    buf = torch.full((n * (c + pad) + shift,), math.nan, dtype=dt, device=DEV)
    x = buf[shift:].view(n, c + pad)[:, :c]
    x.copy_(torch.randn(n, c, generator=gen, device=DEV) * std)
    return x


def finite(x):
    """For the reference: zeros in place of what must not be used."""
    return torch.where(torch.isfinite(x), x, 0)


def case(T, H, V, dtype, pad=0, shift=0, ignored=0.0, bits=64, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[dtype]
    x = rows(gen, T, H, dt, pad, 1.0, shift)
    w = rows(gen, V, H, dt, 0, 2.0 / math.sqrt(max(H, 1)), shift)
    targets = torch.randint(0, V, (T,), generator=gen, device=DEV)
    targets = torch.where(torch.rand(T, generator=gen, device=DEV) < ignored, -100, targets)
    d_loss = torch.rand(T, generator=gen, device=DEV) + 0.5
    return x, w, targets.to(torch.int64 if bits == 64 else torch.int32), d_loss


def run(x, w, targets, d_loss, ignore=-100, scale=1.0, z=0.0):
    print(f"[gpu] cross entropy x={tuple(x.shape)} {x.stride()} w={tuple(w.shape)} {x.dtype} scale={scale} z={z}", flush=True)
    how = dict(ignore_index=ignore, scale=scale, z_loss=z)
    loss, saved = g.linear_cross_entropy(x, w, targets, **how)
    dx, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, **how)
    torch.cuda.synchronize()
    want, err, kept = ref.cross_entropy(finite(x), w, targets, ignore, scale, z)
    check(loss, want, err, "loss")
    for got, (r, e), name in zip((dx, dw), ref.gradients(d_loss, finite(x), w, kept, HALF[x.dtype]), ("dx", "dw")):
        check(got, r, e, name)
    return loss, dx, dw


SMALL = [(1, 8, 1), (1, 64, 7), (3, 72, 300), (5, 4, 33), (2, 1, 10), (32, 136, 129), (33, 200, 257), (64, 520, 1000),
         (65, 512, 777), (130, 264, 1025), (300, 1001, 2049), (257, 64, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,V", SMALL)
def test_sizes(T, H, V, dtype):
    run(*case(T, H, V, dtype))


# tiles of 256 x 256 in every product; two pieces with a tile's K shared and not; many rows of a narrow head
@pytest.mark.parametrize("T,H,V,dtype", [(520, 2048, 22000, "bf16"), (2051, 2056, 8200, "f16"), (2051, 64, 66001, "bf16"),
                                         (16390, 1024, 9001, "bf16")])
def test_large(T, H, V, dtype):
    run(*case(T, H, V, dtype))


@pytest.mark.parametrize("T", [7, 64, 200])
@pytest.mark.parametrize("H,pad,shift", [(64, 3, 0), (64, 8, 0), (61, 0, 0), (72, 0, 1), (72, 8, 8)])
def test_strides_and_alignment(T, H, pad, shift):
    run(*case(T, H, 500, "bf16", pad=pad, shift=shift))


@pytest.mark.parametrize("T", [9, 64, 400])
@pytest.mark.parametrize("bits", [32, 64])
def test_tokens_without_a_label(T, bits):
    x, w, targets, d_loss = case(T, 128, 1000, "bf16", ignored=0.5, bits=bits)
    x[targets == -100] = math.nan
    x[targets == -100, ::2] = math.inf
    loss, dx, dw = run(x, w, targets, d_loss)
    assert bool((dx[targets == -100] == 0).all())


@pytest.mark.parametrize("T", [9, 400])
def test_no_token_has_a_label(T):
    x, w, targets, d_loss = case(T, 128, 1000, "f16")
    targets.fill_(3)
    x.fill_(math.nan)
    loss, saved = g.linear_cross_entropy(x, w, targets, ignore_index=3)
    dx, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, ignore_index=3)
    assert bool((loss == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())


def test_ignore_index_may_be_an_entry():
    x, w, targets, d_loss = case(200, 64, 50, "bf16")
    run(x, w, targets, d_loss, ignore=7)


def test_tokens_whose_loss_has_no_weight():
    x, w, targets, d_loss = case(300, 128, 1000, "bf16")
    d_loss[::3] = 0
    loss, saved = g.linear_cross_entropy(x, w, targets)
    x2 = x.clone()
    x2[::3] = math.nan
    dx, dw = g.linear_cross_entropy_backward(d_loss, x2, w, targets, saved)
    _, _, kept = ref.cross_entropy(x, w, targets, -100, 1.0, 0.0)
    for got, (r, e), name in zip((dx, dw), ref.gradients(d_loss, x, w, kept, HALF[x.dtype]), ("dx", "dw")):
        check(got, r, e, name)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("scale,z", [(0.25, 0.0), (3.0, 0.0), (1.0, 1e-2), (0.5, -1e-3), (1.0, 3000.0)])
def test_scale_and_z_loss(T, scale, z, dtype):
    x, w, targets, d_loss = case(T, 256, 700, dtype)
    run(x, w, targets, d_loss, scale=scale, z=z)


@pytest.mark.parametrize("size", [1e-6, 1e-3, 300.0])
def test_fp16_gradients_of_any_size(size):
    x, w, targets, d_loss = case(100, 128, 3000, "f16")
    d_loss *= size
    d_loss[::2] *= -0.01
    run(x, w, targets, d_loss)


def test_a_confident_head():
    """p of the label near 1: p - 1 keeps its digits, for it is subtracted before it is rounded."""
    x, w, targets, d_loss = case(70, 64, 500, "bf16")
    w[targets] = x * 0.25
    run(x, w, targets, d_loss)


@pytest.mark.parametrize("T", [5, 100])
@pytest.mark.parametrize("bad", [-1, 1000, 1 << 40])
def test_a_label_outside_the_vocabulary_gives_nan(T, bad):
    x, w, targets, d_loss = case(T, 64, 1000, "bf16")
    want = g.linear_cross_entropy(x, w, targets)[0]
    targets[2] = bad
    loss, saved = g.linear_cross_entropy(x, w, targets)
    assert math.isnan(float(loss[2]))
    keep = torch.arange(T, device=DEV) != 2
    assert torch.equal(loss[keep], want[keep])
    dx, _ = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
    assert bool(torch.isnan(dx[2]).all()) and not bool(torch.isnan(dx[keep]).any())


def test_other_values_that_are_not_finite():
    x, w, targets, d_loss = case(100, 64, 1000, "bf16")
    want = g.linear_cross_entropy(x, w, targets)[0]
    x[4, 3], x[5, 0] = math.nan, math.inf
    loss = g.linear_cross_entropy(x, w, targets)[0]
    keep = torch.ones(100, dtype=torch.bool, device=DEV)
    keep[4:6] = False
    assert bool(torch.isnan(loss[4:6]).all()) and torch.equal(loss[keep], want[keep])


def test_sizes_of_zero():
    x, w, targets, d_loss = case(0, 64, 1000, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    dx, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
    assert loss.shape == (0,) and dx.shape == (0, 64) and bool((dw == 0).all())
    x, w, targets, d_loss = case(70, 0, 1000, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    dx, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
    assert float((loss - math.log(1000)).abs().max()) < 1e-5 and dx.shape == (70, 0) and dw.shape == (1000, 0)


def test_one_gradient_alone():
    x, w, targets, d_loss = case(100, 64, 1000, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    both = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
    dx, none = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, need_dw=False)
    assert none is None and torch.equal(dx, both[0])
    none, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, need_dx=False)
    assert none is None and torch.equal(dw, both[1])
    assert g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, need_dx=False, need_dw=False) == (None, None)


# ---- distillation ------------------------------------------------------------------


def teacher(T, V, k, dt=torch.float32, short=0.0, same=False, seed=1, pad=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.randint(0, max(1, V // 8) if same else V, (T, k), generator=gen, device=DEV).int()
    z = (torch.randn(T, k + pad, generator=gen, device=DEV) * 2).to(dt)[:, :k]
    gone = torch.rand(T, k, generator=gen, device=DEV) < short
    return torch.where(gone, -1, ids), z


def run_teacher(x, w, ids, z, d_loss, tau=1.0, scale=1.0):
    print(f"[gpu] distillation x={tuple(x.shape)} w={tuple(w.shape)} entries={ids.shape[1]} {z.dtype} tau={tau}", flush=True)
    how = dict(temperature=tau, scale=scale)
    loss, saved = g.linear_distillation(x, w, ids, z, **how)
    dx, dw = g.linear_distillation_backward(d_loss, x, w, saved, **how)
    torch.cuda.synchronize()
    want, err, kept = ref.distillation(finite(x), w, ids, torch.where(ids < 0, 0, z), tau, scale)
    check(loss, want, err, "loss")
    for got, (r, e), name in zip((dx, dw), ref.gradients(d_loss, finite(x), w, kept, HALF[x.dtype]), ("dx", "dw")):
        check(got, r, e, name)
    return loss, dx, dw


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,V,k", [(1, 64, 300, 1), (4, 72, 300, 3), (40, 256, 1000, 64), (64, 64, 129, 65),
                                     (100, 129, 1025, 20), (300, 520, 3000, 256), (520, 2048, 22000, 64)])
def test_teacher_sizes(T, H, V, k, dtype):
    x, w, _, d_loss = case(T, H, V, dtype)
    run_teacher(x, w, *teacher(T, V, k), d_loss, tau=2.0)


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
def test_teacher_entries(T, dt):
    """Entries that do not exist, twice the same, of no weight; tokens with none."""
    x, w, _, d_loss = case(T, 128, 400, "bf16")
    ids, z = teacher(T, 400, 33, dt, short=0.3, same=True, pad=2)
    z = z.clone()
    z[:, 4] = -math.inf
    ids[3] = -1                     # no entries
    z[5] = -math.inf                # none of any weight
    ids[6, :], z[6, :] = 17, 1.0    # one entry 33 times
    z[ids < 0] = math.nan           # is not read as a value
    x[3], x[5] = math.nan, math.inf
    for tau in (1.0, 4.0):
        loss, dx, _ = run_teacher(x, w, ids, z, d_loss, tau=tau, scale=0.5)
        assert float(loss[3]) == float(loss[5]) == 0 and bool((dx[3] == 0).all()) and bool((dx[5] == 0).all())


@pytest.mark.parametrize("T", [20, 200])
def test_one_entry_is_a_label(T):
    x, w, targets, d_loss = case(T, 128, 400, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    grads = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
    z = torch.full((T, 1), 3.0, device=DEV)
    same, saved = g.linear_distillation(x, w, targets.int().unsqueeze(1), z)
    assert torch.equal(loss, same)
    for a, b in zip(grads, g.linear_distillation_backward(d_loss, x, w, saved)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [20, 200])
def test_teacher_values_that_give_nan(T):
    x, w, _, d_loss = case(T, 64, 300, "bf16")
    ids, z = teacher(T, 300, 9)
    want = g.linear_distillation(x, w, ids, z)[0]
    ids[1, 4], z[2, 8], z[3, 0] = 300, math.nan, math.inf
    loss, saved = g.linear_distillation(x, w, ids, z)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1:4] = False
    assert bool(torch.isnan(loss[1:4]).all()) and torch.equal(loss[keep], want[keep])
    dx, _ = g.linear_distillation_backward(d_loss, x, w, saved)
    assert bool(torch.isnan(dx[1:4]).all()) and not bool(torch.isnan(dx[keep]).any())


# ---- how the calls are used ------------------------------------------------------------


@pytest.mark.parametrize("T,V", [(3, 500), (200, 500), (2051, 66001)])
def test_runs_give_the_same_bits(T, V):
    x, w, targets, d_loss = case(T, 64, V, "bf16")
    def once():
        loss, saved = g.linear_cross_entropy(x, w, targets)
        return (loss, *g.linear_cross_entropy_backward(d_loss, x, w, targets, saved))
    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


@pytest.mark.parametrize("T", [16, 200])
def test_captured_and_replayed(T):
    x, w, targets, d_loss = case(T, 128, 1000, "bf16", ignored=0.2)
    ids, z = teacher(T, 1000, 12)
    def step():
        loss, saved = g.linear_cross_entropy(x, w, targets)
        a = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved)
        other, saved = g.linear_distillation(x, w, ids, z, temperature=2.0)
        return (loss, *a, other, *g.linear_distillation_backward(d_loss, x, w, saved, temperature=2.0))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        y, _, t, d = case(T, 128, 1000, "bf16", ignored=0.3 * seed, seed=10 + seed)
        x.copy_(y), targets.copy_(t), d_loss.copy_(d)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured))


def test_on_another_stream():
    x, w, targets, d_loss = case(200, 128, 1000, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    want = (loss, *g.linear_cross_entropy_backward(d_loss, x, w, targets, saved))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    loss, saved = g.linear_cross_entropy(x, w, targets, stream=s)
    got = (loss, *g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, stream=s))
    del saved
    kept = [torch.full((200,), math.nan, device=DEV) for _ in range(6)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del kept
