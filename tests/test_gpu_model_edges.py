"""The model operators as callers may use them beside the plain cases: through
the C entries with outputs and workspaces that end where they must, two calls
and two graphs at once, orders that no sort made, tensors elsewhere, and drawn
sizes."""
import ctypes
import math
import random

import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import model as m
import model_ref as ref
import test_gpu_experts as experts
import test_gpu_head_loss as head

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def stream():
    return torch.cuda.current_stream().cuda_stream


def guarded(nbytes, lead=256):
    """A buffer of bytes 0xA5 and the address of nbytes inside it."""
    buf = torch.full((lead + nbytes + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, buf.data_ptr() + lead, lead, nbytes


def untouched(g_):
    buf, _, lead, n = g_
    return bool((buf[:lead] == 0xA5).all()) and bool((buf[lead + n:] == 0xA5).all())


@pytest.mark.parametrize("T,H,V,k", [(1, 8, 1, 0), (3, 61, 130, 0), (65, 72, 257, 0), (513, 1001, 2049, 0), (1100, 264, 9000, 0),
                                     (2051, 64, 66001, 0), (4100, 64, 66001, 0), (1, 8, 300, 3), (70, 61, 1000, 9), (600, 520, 4097, 20)])
def test_nothing_behind_the_outputs_is_written(T, H, V, k):
    x, w, targets, d_loss = head.case(T, H, V, "bf16", ignored=0.1)
    print(f"[gpu] guards T={T} H={H} V={V} k={k}", flush=True)
    a = m.gemm_head_args(type=int(g.Dtype.BF16), tokens=T, hidden=H, vocab=V, x=x.data_ptr(), ldx=x.stride(0), w=w.data_ptr(),
                         scale=1.0, z_loss=0.0)
    n = max(k, 1)
    sizes = dict(loss=T * 4, lse=T * 4, picked=T * n * 4, ids=T * n * 4, weights=T * n * 4, mass=T * 4, dx=T * H * 2, dw=V * H * 2)
    if k:
        ids, z = head.teacher(T, V, k)
        a.teacher_ids, a.teacher_logits, a.ld_teacher, a.entries = ids.data_ptr(), z.data_ptr(), z.stride(0), k
        a.teacher_type, a.temperature = int(g.Dtype.F32), 1.0
        assert z.dtype == torch.float32
    else:
        a.targets, a.target_bits, a.ignore_index = targets.data_ptr(), 64, -100
    b = {name: guarded(size) for name, size in sizes.items()}
    saved = m.gemm_head_saved(**{name: b[name][1] for name in ("lse", "picked", "ids", "weights", "mass")})
    for backward in (0, 1):
        need = g.lib.gemm_head_workspace(ctypes.byref(a), backward)
        ws = guarded(need)
        if backward:
            status = g.lib.gemm_head_backward(ctypes.byref(a), d_loss.data_ptr(), ctypes.byref(saved), b["dx"][1], b["dw"][1],
                                              ws[1], need, stream())
        else:
            status = g.lib.gemm_head_loss(ctypes.byref(a), b["loss"][1], ctypes.byref(saved), ws[1], need, stream())
        assert status == 0, g.lib.gemm_last_error()
        torch.cuda.synchronize()
        assert untouched(ws), f"behind the workspace, backward={backward}"
        assert all(untouched(v) for v in b.values()), [name for name, v in b.items() if not untouched(v)]
    if not k:
        loss, s = g.linear_cross_entropy(x, w, targets)
        dx, dw = g.linear_cross_entropy_backward(d_loss, x, w, targets, s)
    else:
        loss, s = g.linear_distillation(x, w, ids, z)
        dx, dw = g.linear_distillation_backward(d_loss, x, w, s)
    for name, t in (("loss", loss), ("dx", dx), ("dw", dw)):
        got = b[name][0][256:256 + sizes[name]]
        assert torch.equal(got, t.contiguous().view(torch.uint8).flatten()), name


def test_nothing_behind_the_rows_is_written():
    T, H, k, E, ld = 77, 61, 3, 9, 70
    ids = experts.choices(T, k, E, 0.2).to(DEV)
    need = g.lib.gemm_expert_sort_workspace(T, k, E)
    off, row_of, ws = guarded((E + 1) * 4), guarded(T * k * 4), guarded(need)
    assert g.lib.gemm_expert_sort(ids.data_ptr(), 64, T, k, E, off[1], row_of[1], ws[1], need, stream()) == 0
    x = torch.randn(T, H, device=DEV)
    rows, d_rows = (torch.full((T * k, ld), 7.0, device=DEV) for _ in range(2))
    out = torch.full((T, ld), 7.0, device=DEV)
    wt, d_wt = torch.rand(T, k, device=DEV), guarded(T * k * 4)
    f32 = int(g.Dtype.F32)
    assert g.lib.gemm_expert_gather(f32, x.data_ptr(), H, rows.data_ptr(), ld, T, H, k, E, off[1], row_of[1], stream()) == 0
    assert g.lib.gemm_expert_combine(f32, rows.data_ptr(), ld, wt.data_ptr(), out.data_ptr(), ld, T, H, k, E, off[1], row_of[1],
                                     stream()) == 0
    assert g.lib.gemm_expert_combine_backward(f32, out.data_ptr(), ld, rows.data_ptr(), ld, wt.data_ptr(), d_rows.data_ptr(), ld,
                                              d_wt[1], T, H, k, E, off[1], row_of[1], stream()) == 0
    torch.cuda.synchronize()
    for t in (rows, d_rows, out):
        assert bool((t[:, H:] == 7).all()) and not bool((t[:, :H] == 7).all(0).any())
    assert all(untouched(v) for v in (off, row_of, ws, d_wt))
    order = g.expert_sort(ids, E)
    assert torch.equal(rows[:, :H], g.expert_gather(x, order))
    assert torch.equal(out[:, :H], g.expert_combine(rows[:, :H], order, wt))


def test_an_order_that_no_sort_made():
    """Rows outside the list are none, and so is what no slot has behind a last
    offset that lies outside it."""
    T, k, H = 5, 2, 70
    row_of = torch.tensor([[0, 10], [-1, 1], [2**31 - 1, 2], [-2**31, 3], [4, 5]], dtype=torch.int32, device=DEV)
    real = (row_of >= 0) & (row_of < T * k)
    x, y, wt = torch.randn(T, H, device=DEV), torch.randn(T * k, H, device=DEV), torch.rand(T, k, device=DEV) + 0.5
    for last in (6, -3, 1000):
        order = g.ExpertOrder(torch.tensor([0, last], dtype=torch.int32, device=DEV), row_of)
        rows = g.expert_gather(x, order)
        out = g.expert_combine(y, order, wt)
        d_rows, d_wt = g.expert_combine_backward(x, y, order, wt)
        at = torch.where(real, row_of, 0).long()
        want = (torch.where(real, wt, 0)[..., None].double() * y[at].double()).sum(1)
        assert torch.allclose(out.double(), want, rtol=0, atol=1e-5)   # two products of some 4 and a sum in fp32
        assert bool((d_wt[~real] == 0).all())
        if last < 0:   # every row is behind it and to be cleared, and six have a slot: the order says both
            continue
        for t, j in real.nonzero().tolist():
            assert torch.equal(rows[row_of[t, j]], x[t]) and torch.equal(d_rows[row_of[t, j]], wt[t, j] * x[t])


def test_tensors_elsewhere_are_refused():
    x, w, targets, d_loss = head.case(5, 64, 100, "bf16")
    loss, saved = g.linear_cross_entropy(x, w, targets)
    for bad in ((x.cpu(), w, targets), (x, w.cpu(), targets), (x, w, targets.cpu())):
        with pytest.raises(ValueError, match="device tensor"):
            g.linear_cross_entropy(*bad)
    for bad in (d_loss.cpu(), *((d_loss, *(s.cpu() if i == j else s for j, s in enumerate(saved))) for i in range(2))):
        d, kept = (bad, saved) if torch.is_tensor(bad) else (bad[0], tuple(bad[1:]))
        with pytest.raises(ValueError, match="device tensor"):
            g.linear_cross_entropy_backward(d, x, w, targets, kept)
    ids, z = head.teacher(5, 100, 4)
    for bad in ((ids.cpu(), z), (ids, z.cpu())):
        with pytest.raises(ValueError, match="device tensor"):
            g.linear_distillation(x, w, *bad)
    choice = torch.zeros(5, 2, dtype=torch.int64, device=DEV)
    order = g.expert_sort(choice, 3)
    with pytest.raises(ValueError, match="device tensor"):
        g.expert_sort(choice.cpu(), 3)
    for bad in (g.ExpertOrder(order.offsets.cpu(), order.row_of), g.ExpertOrder(order.offsets, order.row_of.cpu())):
        with pytest.raises(ValueError, match="device tensor"):
            g.expert_gather(x, bad)
        with pytest.raises(ValueError, match="device tensor"):
            g.expert_combine(x.repeat(2, 1), bad)


def training_step(T, H, V, k, E, seed):
    x, w, targets, d_loss = head.case(T, H, V, "bf16", ignored=0.2, seed=seed)
    ids, z = head.teacher(T, V, 5)
    choice = experts.choices(T, k, E, 0.1, seed=seed).to(DEV)
    wt = torch.rand(T, k, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))

    def step():
        order = g.expert_sort(choice, E)
        rows = g.expert_gather(x, order)
        y = g.expert_combine(rows, order, wt)
        loss, saved = g.linear_cross_entropy(y, w, targets)
        dx, dw = g.linear_cross_entropy_backward(d_loss, y, w, targets, saved)
        other, saved = g.linear_distillation(y, w, ids, z)
        dx2, dw2 = g.linear_distillation_backward(d_loss, y, w, saved)
        d_rows, d_wt = g.expert_combine_backward(dx, rows, order, wt)
        return (loss, dx, dw, other, dx2, dw2, d_rows, d_wt, g.expert_gather_backward(d_rows, order))
    return step


def test_two_streams_at_once():
    steps = [training_step(300, 128, 3001, 4, 8, 0), training_step(70, 264, 1000, 2, 100, 1)]
    want = [s() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, st) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(st):
                got[i].append(s())
    torch.cuda.synchronize()
    for a, runs in zip(want, got):
        for b in runs:
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs():
    """Replayed in turn and at once, with eager calls between."""
    steps = [training_step(300, 128, 3001, 4, 8, 0), training_step(70, 264, 1000, 2, 100, 1)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    graphs, results = [], []
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(s())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in steps]
    for turn in range(4):
        for r in results:
            for t in r:
                t.fill_(7)
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        eager = [s() for s in steps]
        torch.cuda.synchronize()
        for a, b, c in zip(want, results, eager):
            assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c)), turn


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes(seed):
    r = random.Random(seed)
    T = int(math.exp(r.uniform(0, math.log(1500))))
    H, V = int(math.exp(r.uniform(math.log(4), math.log(1200)))), int(math.exp(r.uniform(math.log(2), math.log(9000))))
    dtype = r.choice(["bf16", "f16"])
    x, w, targets, d_loss = head.case(T, H, V, dtype, pad=r.choice([0, 0, 3, 8]), ignored=r.choice([0.0, 0.3]), seed=seed)
    head.run(x, w, targets, d_loss, scale=r.choice([1.0, 0.3]), z=r.choice([0.0, 1e-3]))
    head.run_teacher(x, w, *head.teacher(T, V, r.randint(1, min(V, 100))), d_loss, tau=r.choice([1.0, 3.0]))


# a vocabulary in two pieces: a tile's K shared and not, 128 and 256 wide
@pytest.mark.parametrize("T,H,V,dtype", [(4100, 64, 66001, "bf16"), (16390, 1024, 17001, "bf16"), (4100, 1024, 66001, "f16")])
def test_pieces(T, H, V, dtype):
    x, w, targets, d_loss = head.case(T, H, V, dtype, ignored=0.2)
    dx, dw = head.run(x, w, targets, d_loss, z=1e-4)[1:]
    how = dict(z_loss=1e-4)
    loss, saved = g.linear_cross_entropy(x, w, targets, **how)
    again = g.linear_cross_entropy_backward(d_loss, x, w, targets, saved, **how)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_pieces_from_a_teacher():
    x, w, _, d_loss = head.case(4100, 136, 66001, "bf16")
    head.run_teacher(x, w, *head.teacher(4100, 66001, 30), d_loss, tau=2.0)


# rows counted by a launch of their own
@pytest.mark.parametrize("T", [4096, 4097, 5120, 20001, 70000])
def test_many_tokens(T):
    x, w, targets, d_loss = head.case(T, 72, 300, "f16", ignored=0.4)
    x[targets == -100] = math.nan
    d_loss[::7] = 0
    head.run(x, w, targets, d_loss, z=1e-3)


def test_many_tokens_of_which_few_have_a_label():
    x, w, targets, d_loss = head.case(9000, 64, 500, "bf16")
    keep = torch.zeros(9000, dtype=torch.bool, device=DEV)
    keep[[1023, 1024, 8999]] = True
    targets[~keep] = -100
    head.run(x, w, targets, d_loss)
    targets[:] = -100
    loss, dx, dw = head.run(x, w, targets, d_loss)
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("T,k,E", [(4096, 1, 64), (4097, 1, 64), (2048, 2, 1024), (1025, 4, 3), (65536, 4, 300), (262145, 1, 7)])
def test_order_in_parts(T, k, E):
    experts.test_order(T, k, E, torch.int64)


def test_more_rows_than_a_launch_holds():
    """17 million tokens of one element: 2^32 threads are not one launch."""
    T = (1 << 24) + 100
    free, _ = torch.cuda.mem_get_info()
    if free < 8 << 30:
        pytest.skip("memory")
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(T, 1, generator=gen, device=DEV).half()
    order = g.expert_sort(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1)
    at = torch.arange(T, dtype=torch.int32, device=DEV)[:, None]
    assert torch.equal(order.row_of, at) and order.bounds() == [0, T]
    assert torch.equal(g.expert_gather(x, order), x) and torch.equal(g.expert_combine(x, order), x)
    w = torch.rand(T, 1, generator=gen, device=DEV)
    d_rows, d_w = g.expert_combine_backward(x, x, order, w)
    # The product of 11 and 24 bits is exact in 64; it is rounded to fp16 (half a step, 2^-11 of it or 2^-25) at once or
    # after a rounding to fp32 (2^-24 of it), which do not always give the same number.
    want = x.double() * w
    assert float(((d_rows.double() - want).abs() - want.abs() * (2**-11 + 2**-24) - 2**-25).max()) <= 0
    assert torch.equal(d_w, x.float() * x.float())


def test_a_loss_of_the_most_tokens():
    """The largest number of tokens: two entries whose logits are 0 and x."""
    T = (1 << 26) - 64
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("memory")
    x = torch.zeros(T, 8, dtype=torch.float16, device=DEV)
    x[:, 0] = torch.arange(T, device=DEV) % 8 - 4
    w = torch.zeros(2, 8, dtype=torch.float16, device=DEV)
    w[1, 0] = 1
    targets = torch.ones(T, dtype=torch.int32, device=DEV)
    targets[::3] = -100
    loss, _ = g.linear_cross_entropy(x, w, targets)
    values = torch.arange(8, device=DEV).double() - 4
    # exp, log and their sum in fp32: a few 2^-23 of values below 5
    want = torch.nn.functional.softplus(-values)
    for r in range(8):
        mine = loss[r::8]
        learn = targets[r::8] != -100
        assert not bool(mine[~learn].any())
        assert float((mine[learn].double() - want[r]).abs().max()) <= 8 * 5 * 2**-23
