"""MXFP4 quantiser, its inverse, and the linear layer with its gradients,
against the 64-bit forms of block_ref."""
import pytest
import torch

import dense_gemm_epilogue_02_amd as g
import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def draw(rows, cols, dtype, seed, pad=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=gen) * std
    return x.to(TYPES[dtype])[:, :cols]


def check_form(q, x, what):
    """An Mx4 against the reference of x quantised along its rows, padding included."""
    v, byte = ref.quantize(x)
    R, k = x.shape
    assert q.rows == R and q.k == k
    sc, nb = q.scales.cpu(), byte.shape[1]
    assert torch.equal(sc[:, :nb], byte), f"{what}: scale bytes"
    assert bool((sc[:, nb:] == 127).all()), f"{what}: padding scales"
    got = ref.unpack(q.codes, q.scales, q.codes.shape[1] * 2)
    assert torch.equal(torch.nan_to_num(got[:, :k], nan=7e9), torch.nan_to_num(v, nan=7e9)), f"{what}: values"
    # codes past k stand for zero (in a short last block they share its scale)
    assert bool((got[:, nb * 32:] == 0).all()), f"{what}: padding codes"
    tail = ref.unpack(q.codes, torch.full_like(q.scales, 127), q.codes.shape[1] * 2)[:, k:]
    assert bool((tail == 0).all()), f"{what}: codes past the end"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 1), (128, 128, 0), (130, 257, 3),
                                           (31, 1000, 8), (300, 129, 0), (5, 2049, 7)])
def test_quantize_both(rows, cols, pad, dtype):
    x = draw(rows, cols, dtype, rows * 7 + cols, pad)
    x[:, ::17] *= 100
    buf = torch.empty(rows, cols + pad, dtype=x.dtype, device=DEV)
    buf[:, :cols] = x.to(DEV)
    xd = buf[:, :cols]
    print(f"[gpu] quantize {rows}x{cols}+{pad} {dtype}", flush=True)
    a, b = g.mx4_quantize(xd, "both")
    check_form(a, x, "rows")
    check_form(b, x.t(), "columns")
    a1, b0 = g.mx4_quantize(xd, 1), g.mx4_quantize(xd, 0)
    for p, q in ((a, a1), (b, b0)):
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    v, _ = ref.quantize(x)
    assert torch.equal(g.mx4_dequantize(a).cpu().double(), v)
    for t in TYPES.values():
        assert torch.equal(g.mx4_dequantize(a, t).cpu(), v.to(t))


def test_quantize_borders_and_extremes():
    """Ties of every border, the saturating range, blocks of zeros, subnormal
    blocks, the largest values, and NaN / infinities that spoil one block only."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 4.0])
    row = torch.zeros(14, 96)
    row[0, :11], row[1, :11] = ties, -ties
    row[2, 32:43] = ties * 2.0 ** 100
    row[3, :11] = ties * 2.0 ** -120
    row[4, :3] = torch.tensor([1e-40, 3e-41, -1e-45])       # fp32 subnormals
    row[5, :2] = torch.tensor([3.4e38, -1e38])
    row[6, 40] = float("nan")
    row[7, 3] = float("inf")
    row[8, 70] = -float("inf")
    row[9, :32] = -0.0
    row[10, :32] = 2.0 ** -126 * torch.arange(32)
    row[11, :32] = 2.0 ** -128 * torch.arange(32)
    row[12, ::32] = torch.tensor([1.0, 2.0, 4.0])
    row[13, :32] = torch.nextafter(ties[:1], torch.tensor([1.0])).expand(32) * 4
    for scale, dtype in ((1.0, torch.float32), (1.0, torch.bfloat16)):
        x = (row * scale).to(dtype)
        print(f"[gpu] quantize extremes {dtype}", flush=True)
        a, b = g.mx4_quantize(x.to(DEV), "both")
        check_form(a, x, "rows")
        check_form(b, x.t(), "columns")
        v, _ = ref.quantize(x)
        got = g.mx4_dequantize(a).cpu().double()
        assert torch.equal(torch.nan_to_num(got, nan=7e9), torch.nan_to_num(v, nan=7e9))


def test_quantize_follows_synthetic_generator():
    """The codes that the MX GEMM tests are fed with are the same ones."""
    import synthetic as syn
    x = draw(64, 512, "f32", 3)
    q = g.mx4_quantize(x.to(DEV), 1)
    codes, scales = syn.mx4_quantize_device(x.to(DEV))
    assert torch.equal(q.scales, scales)
    assert torch.equal(ref.unpack(q.codes, q.scales, 512), ref.unpack(codes, scales, 512))


def run_linear(M, N, K, dtype, bias, pad, seed, act="linear"):
    x, w = draw(M, K, dtype, seed, pad), draw(N, K, "bf16", seed + 1, 0, 0.05)
    codes, scales, wv = ref.pack(w)
    b = draw(1, N, "bf16", seed + 2)[0] if bias else None
    layer = g.Mx4Linear(g.Mx4(codes.to(DEV), scales.to(DEV), K), activation=act)
    buf = torch.full((M, K + pad), float("nan"), dtype=x.dtype, device=DEV)
    buf[:, :K] = x.to(DEV)
    guard = torch.full((M + 2, N), 77.0, dtype=torch.bfloat16, device=DEV)
    print(f"[gpu] linear M={M} N={N} K={K} {dtype} bias={bias} pad={pad} {act}", flush=True)
    y = layer.forward(buf[:, :K], None if b is None else b.to(DEV), out=guard[1:-1])
    torch.cuda.synchronize()
    assert bool((guard[0] == 77).all()) and bool((guard[-1] == 77).all()), "wrote outside y"
    xv, _ = ref.quantize(x)
    r, e = ref.matmul_bound(xv, wv, 0.0)
    if b is not None:
        r = r + b.double()
        e = e + ref.F32 * r.abs()
    if act == "relu":
        r = r.clamp_min(0)
    ref.check(y, r, e + 2.0 ** -8 * r.abs(), "y")
    layer.close()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 65, 200])
@pytest.mark.parametrize("N,K", [(1, 32), (33, 100), (128, 256), (257, 1056)])
def test_linear_sizes(M, N, K):
    run_linear(M, N, K, "bf16", M % 2 == 0, 3 * (M % 3), M * 1000 + N)


@pytest.mark.parametrize("M,N,K", [(65, 257, 2048), (65, 257, 2049), (321, 6001, 256), (1024, 2049, 300), (1025, 2040, 300)])
def test_linear_between_tiles(M, N, K):
    """Both sides of the lengths and of the number of tiles where the tile changes."""
    run_linear(M, N, K, "bf16", True, 0, M + K)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(1, 64, 2048, 0), (20, 100, 511, 5), (70, 64, 300, 1)])
def test_linear_types(M, N, K, pad, dtype):
    run_linear(M, N, K, dtype, True, pad, 5)


@pytest.mark.parametrize("M", [4, 40])
def test_linear_activation(M):
    run_linear(M, 96, 320, "bf16", True, 0, 9, "relu")


def test_linear_empty():
    w = g.mx4_quantize(torch.ones(40, 64, device=DEV), 1)
    layer = g.Mx4Linear(w)
    assert layer.forward(torch.empty(0, 64, device=DEV)).shape == (0, 40)
    for M in (3, 50):   # K == 0: the bias alone
        w0 = g.Mx4(torch.empty(40, 0, dtype=torch.uint8, device=DEV), torch.empty(40, 0, dtype=torch.uint8, device=DEV), 0)
        b = torch.arange(40, dtype=torch.bfloat16, device=DEV)
        y = g.Mx4Linear(w0).forward(torch.empty(M, 0, device=DEV), b)
        assert torch.equal(y, b.expand(M, 40))


def test_linear_nan_stays_in_its_row():
    """A NaN in x spoils its row of y and no other; a NaN block of W its column."""
    for M in (3, 40):
        x, w = draw(M, 128, "bf16", 1), draw(48, 128, "bf16", 2)
        x[1, 5] = float("nan")
        q = g.mx4_quantize(w.to(DEV), 1)
        q.scales[7, 2] = 255
        y = g.Mx4Linear(q).forward(x.to(DEV)).cpu()
        nan = torch.zeros(M, 48, dtype=torch.bool)
        nan[1], nan[:, 7] = True, True
        assert torch.equal(torch.isnan(y), nan)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(1, 1, 1, 0), (2, 33, 64, 0), (32, 64, 32, 8), (100, 130, 70, 3), (257, 96, 300, 0)])
def test_backward(M, N, K, pad, dtype):
    dy, x, w = draw(M, N, dtype, 1, pad, 0.01), draw(M, K, dtype, 2, pad), draw(N, K, "bf16", 3, 0, 0.05)
    dyd, xd = (torch.nn.functional.pad(t, (0, pad)).to(DEV)[:, :t.shape[1]] for t in (dy, x))
    layer = g.Mx4Linear.from_weight(w.to(DEV), backward=True)
    print(f"[gpu] backward M={M} N={N} K={K} {dtype} pad={pad}", flush=True)
    dx, dw = layer.backward(dyd, xd)
    wt, _ = ref.quantize(w.t())
    r, e = ref.matmul_bound(ref.quantize(dy)[0], wt, 2.0 ** -8)
    ref.check(dx, r, e, "dx")
    r, e = ref.matmul_bound(ref.quantize(dy.t())[0], ref.quantize(x.t())[0], 2.0 ** -8)
    ref.check(dw, r, e, "dw")
    only, none = layer.backward(dyd, None, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = layer.backward(dyd, xd, need_dx=False)
    assert none is None and torch.equal(only, dw)


def test_backward_is_the_gradient_where_nothing_rounds():
    """On values that MXFP4 holds exactly, y is linear in x and W, so the
    difference quotient of <dy, y> along any direction is exact."""
    gen = torch.Generator().manual_seed(0)
    M, N, K = 40, 64, 96
    pick = lambda *s: torch.randint(-3, 4, s, generator=gen).double()  # noqa: E731
    dy, x, w, vx, vw = pick(M, N), pick(M, K), pick(N, K), pick(M, K), pick(N, K)
    for t in (dy, x, w):   # a 4 in every block of either direction fixes the scale at 1
        t[::32, :], t[:, ::32] = 4, 4
    loss = lambda x, w: float((dy * (x @ w.t())).sum())  # noqa: E731
    layer = g.Mx4Linear.from_weight(w.float().to(DEV), backward=True)
    dx, dw = layer.backward(dy.float().to(DEV), x.float().to(DEV))
    for got, v, diff in ((dx, vx, loss(x + vx, w) - loss(x, w)), (dw, vw, loss(x, w + vw) - loss(x, w))):
        g64 = got.cpu().double()
        assert abs(float((g64 * v).sum()) - diff) <= 2.0 ** -8 * float((g64 * v).abs().sum())


def test_backward_empty():
    layer = g.Mx4Linear.from_weight(torch.ones(32, 64, device=DEV), backward=True)
    dx, dw = layer.backward(torch.empty(0, 32, device=DEV), torch.empty(0, 64, device=DEV))
    assert dx.shape == (0, 64) and dw.shape == (32, 64) and not bool(dw.any())


def test_linear_on_another_stream_and_repeatable():
    x, w = draw(200, 512, "bf16", 1).to(DEV), draw(300, 512, "bf16", 2).to(DEV)
    layer = g.Mx4Linear.from_weight(w)
    y = layer.forward(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = layer.forward(x, stream=s)
    s.synchronize()
    assert torch.equal(y, z)
