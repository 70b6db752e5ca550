"""The feed-forward block's operators where no GPU is needed: the exports of
include/gemm_block.h, every refusal of the C entries (none of these calls gets
as far as a launch), what the sizes of workspaces promise, the binding's own
checks, and the tests' 64-bit forms against closed forms."""
import ctypes
import os
import re

import pytest
import torch

import dense_gemm_epilogue_02_amd as g
from dense_gemm_epilogue_02_amd import block as b
import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L, S, D = g.lib, g.Status, g.Dtype
P = 1 << 20          # stands for a device address: nothing here reads it
F32, F16, BF16, F8, F4 = (int(t) for t in (D.F32, D.F16, D.BF16, D.F8_E4M3, D.F4_E2M1))


def message():
    return L.gemm_last_error().decode()


def test_every_declared_function_is_bound():
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", txt))
    assert len(names) == 13
    for n in names:
        assert getattr(L, n).argtypes is not None, n


# ---- MXFP4 ----------------------------------------------------------------------


def test_padded():
    assert [g.gemm_mx4_padded(k) for k in (-3, 0, 1, 256, 257, 2 ** 33)] == [0, 0, 256, 256, 512, 2 ** 33]


QUANT = dict(x=P, t=BF16, R=4, C=64, ld=64, rc=P, rs=P, cc=None, cs=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(t=F8), S.UNSUPPORTED, "F32, F16 or BF16"), (dict(R=-1), S.INVALID_ARG, "negative"),
    (dict(C=1 << 31, ld=1 << 31), S.UNSUPPORTED, "2^31"), (dict(x=None), S.INVALID_ARG, "x is NULL"),
    (dict(ld=63), S.INVALID_ARG, "leading dimension"), (dict(ld=1 << 45), S.UNSUPPORTED, "2^46"),
    (dict(x=P + 1), S.INVALID_ARG, "aligned"), (dict(rs=None), S.INVALID_ARG, "go together"),
    (dict(cc=P), S.INVALID_ARG, "go together"), (dict(rc=None, rs=None), S.INVALID_ARG, "neither"),
    (dict(rc=P + 8), S.INVALID_ARG, "16-byte"), (dict(rs=P + 4), S.INVALID_ARG, "8-byte"),
    (dict(cc=P, cs=P + 2), S.INVALID_ARG, "column form")])
def test_quantize_refuses(change, status, word):
    a = {**QUANT, **change}
    assert L.gemm_mx4_quantize(*a.values(), None) == status
    assert word in message()


def test_empty_needs_no_pointers():
    assert L.gemm_mx4_quantize(None, F32, 0, 64, 64, None, None, None, None, None) == 0
    assert L.gemm_mx4_dequantize(None, None, 5, 0, None, F32, 0, None) == 0


def test_dequantize_refuses():
    for args, word in (((None, P, 2, 32, P, F32, 32, None), "NULL"), ((P, P, 2, 32, None, F32, 32, None), "out is NULL"),
                       ((P, P, 2, 32, P, F8, 32, None), "F32"), ((P, P, 2, 32, P, F16, 31, None), "leading"),
                       ((P + 4, P, 2, 32, P, F16, 32, None), "16-byte")):
        assert L.gemm_mx4_dequantize(*args) != 0
        assert word in message()


@pytest.fixture(scope="module")
def plans():
    p = {n: g.Plan("f4e2m1", la="row", lb="col", lc="row", activation=n) for n in ("linear", "relu")}
    p["f16"] = g.Plan("f16", la="row", lb="col", lc="row")
    yield p
    for q in p.values():
        q.close()


LIN = dict(plan=None, x=P, t=BF16, ldx=64, wc=P, ws=P, bias=None, y=P, M=4, N=8, K=64, w=None, wb=0)


@pytest.mark.parametrize("change,status,word", [
    (dict(plan=None), S.NOT_INITIALIZED, "plan"), (dict(plan="f16"), S.UNSUPPORTED, "F4_E2M1"),
    (dict(t=F4), S.UNSUPPORTED, "x must be"), (dict(x=None), S.INVALID_ARG, "x is NULL"),
    (dict(ldx=8), S.INVALID_ARG, "leading"), (dict(y=None), S.INVALID_ARG, "y is NULL"),
    (dict(ws=None), S.INVALID_ARG, "weight"), (dict(bias=P + 1), S.INVALID_ARG, "bias"),
    (dict(M=100), S.INVALID_ARG, "workspace"), (dict(M=100, w=P + 4, wb=1 << 20), S.INVALID_ARG, "16-byte"),
    (dict(M=100, w=P, wb=100), S.INVALID_ARG, "workspace of 100"), (dict(N=-1), S.INVALID_ARG, "negative")])
def test_linear_refuses(plans, change, status, word):
    a = {**LIN, "plan": "linear", **change}
    a["plan"] = plans[a["plan"]].handle if isinstance(a["plan"], str) else a["plan"]
    assert L.gemm_mx4_linear(*a.values(), None) == status
    assert word in message()


def test_linear_backward_refuses(plans):
    base = dict(plan=plans["linear"].handle, dy=P, ldy=8, x=P, ldx=64, t=BF16, wc=P, ws=P, dx=P, dw=P, M=4, N=8, K=64,
                w=P, wb=1 << 30)
    for change, word in ((dict(plan=plans["relu"].handle), "LINEAR"), (dict(dy=None), "dy is NULL"), (dict(x=None), "x is NULL"),
                         (dict(wc=None), "weight"), (dict(K=-2), "negative"), (dict(ldy=3), "leading"),
                         (dict(wb=10), "workspace of 10"), (dict(t=F8), "F32")):
        assert L.gemm_mx4_linear_backward(*{**base, **change}.values(), None) != 0
        assert word in message(), (change, message())
    assert L.gemm_mx4_linear_backward(*{**base, "dx": None, "dw": None, "w": None}.values(), None) == 0


def test_linear_workspaces():
    few = [L.gemm_mx4_linear_workspace(m, 512) for m in range(0, 9)]
    assert few == [0] * 9
    sizes = [L.gemm_mx4_linear_workspace(m, 512) for m in range(9, 200, 7)]
    assert sizes == sorted(sizes) and sizes[0] >= 9 * (256 + 16)
    assert L.gemm_mx4_linear_workspace(100, 0) == 0
    # dy in both directions and x along M
    assert L.gemm_mx4_linear_backward_workspace(256, 512, 1024) >= (256 * 512 * 2 + 1024 * 256) * 17 // 32
    assert L.gemm_mx4_linear_backward_workspace(0, 512, 1024) == 0


# ---- mixture of experts -----------------------------------------------------------


def moe(**kw):
    d = dict(hidden=64, inner=32, experts=8, top_k=2, renormalize=1, type=BF16, weight_type=BF16, router=P, up=P,
             up_scales=None, down=P, down_scales=None)
    return b.gemm_moe_desc(*{**d, **kw}.values())


def run_moe(desc, T=4, ldx=64, x=P, out=P, ldo=64, ids=None, probs=None, ws=P, wsb=1 << 40):
    return L.gemm_moe_forward(desc and ctypes.byref(desc), x, ldx, None, out, ldo, ids, probs, T, ws, wsb, None)


@pytest.mark.parametrize("desc,call,status,word", [
    (dict(hidden=-1), {}, S.INVALID_ARG, "bad size"), (dict(experts=0), {}, S.INVALID_ARG, "bad size"),
    (dict(top_k=9), {}, S.INVALID_ARG, "top_k = 9 of 8"), (dict(experts=513), {}, S.UNSUPPORTED, "512"),
    (dict(experts=64, top_k=17), {}, S.UNSUPPORTED, "16"), ({}, dict(T=65), S.UNSUPPORTED, "at most 64"),
    (dict(inner=(1 << 18) + 1), {}, S.UNSUPPORTED, "above"), (dict(type=F32, weight_type=F32), {}, S.UNSUPPORTED, "F16 or BF16"),
    (dict(weight_type=F16), {}, S.UNSUPPORTED, "weights"), (dict(type=F16, weight_type=F4), {}, S.UNSUPPORTED, "F4_E2M1"),
    ({}, dict(x=None), S.INVALID_ARG, "x is NULL"), ({}, dict(out=None), S.INVALID_ARG, "out is NULL"),
    ({}, dict(ldx=63), S.INVALID_ARG, "leading"), ({}, dict(ldx=1 << 30), S.UNSUPPORTED, "2^31 bytes"),
    (dict(router=None), {}, S.INVALID_ARG, "router"), (dict(up=None), {}, S.INVALID_ARG, "up is NULL"),
    (dict(down=P + 1), {}, S.INVALID_ARG, "down"), (dict(weight_type=F4), {}, S.INVALID_ARG, "scales of up"),
    (dict(weight_type=F4, up_scales=P), {}, S.INVALID_ARG, "scales of down"),
    ({}, dict(ids=P + 2), S.INVALID_ARG, "ids"), ({}, dict(ws=None), S.INVALID_ARG, "workspace"),
    ({}, dict(wsb=64), S.INVALID_ARG, "workspace of 64")])
def test_moe_refuses(desc, call, status, word):
    assert run_moe(moe(**desc), **call) == status
    assert word in message()


def test_moe_null_and_empty():
    assert run_moe(None) == S.INVALID_ARG
    assert run_moe(moe(), T=0, x=None, out=None, ws=None) == 0


def test_moe_workspace_grows_with_the_tokens():
    for E, k in ((4, 1), (8, 8), (64, 6), (512, 16)):
        d = moe(experts=E, top_k=k)
        sizes = [L.gemm_moe_workspace(ctypes.byref(d), t) for t in range(65)]
        assert sizes == sorted(sizes) and 0 < L.gemm_moe_state_bytes(ctypes.byref(d)) <= sizes[0] + 16
        # h's two numbers of every slot at least
        assert sizes[64] >= 64 * k * 32 * 4
    bad = moe(experts=0)
    assert L.gemm_moe_workspace(ctypes.byref(bad), 4) < 0 and L.gemm_moe_state_bytes(ctypes.byref(bad)) < 0


# ---- norms ------------------------------------------------------------------------


def norm(**kw):
    d = dict(type=BF16, gate_act=0, rows=6, cols=64, gate_rows=0, eps=1e-6, block=P, residual=P, gate=None, ld_block=64,
             ld_residual=64, ld_gate=0, w_post=P, scale=P, w_next=P, out=P, next=P, ld_out=64, ld_next=64,
             rstd_post=P, rstd_next=P)
    return b.gemm_norm_args(*{**d, **kw}.values())


@pytest.mark.parametrize("change,status,word", [
    (dict(type=F4), S.UNSUPPORTED, "type"), (dict(rows=-1), S.INVALID_ARG, "negative"),
    (dict(rows=1 << 31), S.UNSUPPORTED, "2^31"), (dict(cols=16385), S.UNSUPPORTED, "16384"),
    (dict(gate_act=1), S.UNSUPPORTED, "gate_act"), (dict(gate=P, gate_rows=4, ld_gate=64), S.INVALID_ARG, "divide"),
    (dict(gate=P, gate_rows=0), S.INVALID_ARG, "divide"), (dict(gate=P, gate_rows=3, ld_gate=8), S.INVALID_ARG, "gate"),
    (dict(block=None), S.INVALID_ARG, "belong to a block"), (dict(block=None, w_post=None, scale=None, w_next=None), S.INVALID_ARG, "neither"),
    (dict(residual=None), S.INVALID_ARG, "residual"), (dict(ld_block=32), S.INVALID_ARG, "block"),
    (dict(out=None), S.INVALID_ARG, "out"), (dict(next=None), S.INVALID_ARG, "next"),
    (dict(w_post=P + 1), S.INVALID_ARG, "w_post"), (dict(scale=P + 1), S.INVALID_ARG, "scale"),
    (dict(w_next=P + 1), S.INVALID_ARG, "w_next"), (dict(rstd_post=P + 2), S.INVALID_ARG, "rstd")])
def test_norm_refuses(change, status, word):
    assert L.gemm_norm_residual(ctypes.byref(norm(**change)), None) == status
    assert word in message()


def norm_back(**kw):
    d = dict(type=F32, gate_act=0, rows=6, cols=64, gate_rows=3, d_out=P, d_next=P, block=P, out=P, gate=P, ld_d_out=64,
             ld_d_next=64, ld_block=64, ld_out=64, ld_gate=64, w_post=P, scale=P, w_next=P, rstd_post=P, rstd_next=P,
             d_block=P, d_residual=P, ld_d_block=64, ld_d_residual=64, d_gate=P, d_scale=P, d_w_post=P, d_w_next=P,
             workspace=P, workspace_bytes=1 << 30)
    return b.gemm_norm_backward_args(*{**d, **kw}.values())


@pytest.mark.parametrize("change,word", [
    (dict(cols=20000), "16384"), (dict(gate_rows=4), "divide"), (dict(block=None), "belong to a block"),
    (dict(w_post=None), "not there"), (dict(gate=None), "not there"), (dict(scale=None), "not there"),
    (dict(w_next=None), "not there"), (dict(d_next=None), "go together"), (dict(d_residual=None), "d_residual"),
    (dict(d_block=None), "d_block"), (dict(out=None), "out"), (dict(rstd_next=None), "rstd"), (dict(rstd_post=P + 1), "rstd"),
    (dict(d_gate=P + 1), "d_gate"), (dict(workspace=None), "workspace"), (dict(workspace_bytes=16), "workspace of 16")])
def test_norm_backward_refuses(change, word):
    assert L.gemm_norm_residual_backward(ctypes.byref(norm_back(**change)), None) != 0
    assert word in message()


def test_null_args():
    for f in (L.gemm_norm_residual, L.gemm_norm_residual_backward):
        assert f(None, None) == S.INVALID_ARG
    assert L.gemm_norm_backward_workspace(None) < 0


@pytest.mark.parametrize("rows,gate_rows", [(0, 0), (1, 1), (7, 7), (1000, 1), (5000, 5000), (6000, 3), (4096, 512)])
def test_norm_backward_workspace_holds_the_parts(rows, gate_rows):
    """Three rows of partial sums a part at least, and never more parts than rows."""
    n = L.gemm_norm_backward_workspace(ctypes.byref(norm_back(rows=rows, gate_rows=gate_rows, cols=128, ld_gate=128)))
    assert n % 16 == 0 and 0 <= n <= 4 * max(rows, 1) * 128 * 4
    assert rows == 0 or n >= 3 * 128 * 4


# ---- the binding's checks ------------------------------------------------------------


def test_binding_refuses_host_tensors_and_bad_words():
    x = torch.ones(4, 32)
    for call in (lambda: g.mx4_quantize(x), lambda: g.norm_residual(None, x), lambda: g.mx4_dequantize(
            g.Mx4(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8), 32)),
            lambda: g.MoeLayer(x.half(), x, x, 1)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="axis"):
        g.mx4_quantize(x, 2)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        g.mx4_quantize(x.int())
    with pytest.raises(ValueError, match="weight"):
        g.Mx4Linear(None)


def test_mx4_shapes():
    c, s = torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(3, 8, dtype=torch.uint8)
    assert g.Mx4(c, s, 200).rows == 3
    for bad in ((c[:, :64], s, 200), (c, s, 300), (c, s[:2], 200), (c.int(), s, 200), (c.t(), s, 200)):
        with pytest.raises(ValueError):
            g.Mx4(*bad)


# ---- the 64-bit forms -------------------------------------------------------------------


def test_reference_quantiser_on_closed_forms():
    v, byte = ref.quantize(torch.tensor([[6.0, 5.0, 2.5, 0.25, -0.75] + [0.0] * 27]))
    assert byte.tolist() == [[127]] and v[0, :5].tolist() == [6.0, 4.0, 2.0, 0.0, -1.0]   # ties to the even code
    v, byte = ref.quantize(torch.tensor([[7.9] + [0.0] * 31 + [8.0] + [0.0] * 31]))
    assert byte.tolist() == [[127, 128]] and v[0, 0] == 6.0 and v[0, 32] == 8.0            # saturated; the next scale
    c, s, w = ref.pack(torch.randn(5, 70, generator=torch.Generator().manual_seed(0)))
    assert torch.equal(ref.unpack(c, s, 70), w)


def test_reference_route_orders_ties_and_nan():
    x = torch.tensor([[1.0, 0.0]])
    router = torch.tensor([[2.0, 0.0], [3.0, 0.0], [float("nan"), 0.0], [3.0, 0.0]])
    ids, p = ref.route(x, router, 3, True)
    assert ids.tolist() == [[1, 3, 0]]
    assert torch.allclose(p.sum(1), torch.ones(1, dtype=torch.float64))
