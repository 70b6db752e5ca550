"""Binding of the feed-forward block's operators (``include/gemm_block.h``):
MXFP4 operands and the linear layer on them, the mixture-of-experts layer for a
few tokens, and the norms around a block.

Argument marshalling only. Tensors are 2-D device tensors whose rows are
contiguous (any distance between rows). Results and workspaces are allocated by
torch on the stream that the kernels are enqueued on (torch's current one,
unless ``stream`` is given). Nothing here takes part in autograd: the backward
passes are calls of their own.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import Dtype, Epilogue, GemmError, Plan, Status, _check, lib

_i32, _i64, _f32, _vp, _st = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                              ctypes.c_int)


class gemm_moe_desc(ctypes.Structure):
    _fields_ = [("hidden", _i64), ("inner", _i64), ("experts", _i32), ("top_k", _i32),
                ("renormalize", _i32), ("type", _st), ("weight_type", _st), ("router", _vp),
                ("up", _vp), ("up_scales", _vp), ("down", _vp), ("down_scales", _vp)]


class gemm_norm_args(ctypes.Structure):
    _fields_ = [("type", _st), ("gate_act", _st), ("rows", _i64), ("cols", _i64),
                ("gate_rows", _i64), ("eps", _f32), ("block", _vp), ("residual", _vp),
                ("gate", _vp), ("ld_block", _i64), ("ld_residual", _i64), ("ld_gate", _i64),
                ("w_post", _vp), ("scale", _vp), ("w_next", _vp), ("out", _vp), ("next", _vp),
                ("ld_out", _i64), ("ld_next", _i64), ("rstd_post", _vp), ("rstd_next", _vp)]


class gemm_norm_backward_args(ctypes.Structure):
    _fields_ = [("type", _st), ("gate_act", _st), ("rows", _i64), ("cols", _i64),
                ("gate_rows", _i64), ("d_out", _vp), ("d_next", _vp), ("block", _vp),
                ("out", _vp), ("gate", _vp), ("ld_d_out", _i64), ("ld_d_next", _i64),
                ("ld_block", _i64), ("ld_out", _i64), ("ld_gate", _i64), ("w_post", _vp),
                ("scale", _vp), ("w_next", _vp), ("rstd_post", _vp), ("rstd_next", _vp),
                ("d_block", _vp), ("d_residual", _vp), ("ld_d_block", _i64),
                ("ld_d_residual", _i64), ("d_gate", _vp), ("d_scale", _vp), ("d_w_post", _vp),
                ("d_w_next", _vp), ("workspace", _vp), ("workspace_bytes", _i64)]


_P = ctypes.POINTER
for _name, _res, _args in (
        ("gemm_mx4_padded", _i64, [_i64]),
        ("gemm_mx4_quantize", _st, [_vp, _st, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
        ("gemm_mx4_dequantize", _st, [_vp, _vp, _i64, _i64, _vp, _st, _i64, _vp]),
        ("gemm_mx4_linear_workspace", _i64, [_i64, _i64]),
        ("gemm_mx4_linear", _st, [_vp, _vp, _st, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp,
                                  _i64, _vp]),
        ("gemm_mx4_linear_backward_workspace", _i64, [_i64, _i64, _i64]),
        ("gemm_mx4_linear_backward", _st, [_vp, _vp, _i64, _vp, _i64, _st, _vp, _vp, _vp, _vp,
                                           _i64, _i64, _i64, _vp, _i64, _vp]),
        ("gemm_moe_state_bytes", _i64, [_P(gemm_moe_desc)]),
        ("gemm_moe_workspace", _i64, [_P(gemm_moe_desc), _i64]),
        ("gemm_moe_forward", _st, [_P(gemm_moe_desc), _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64,
                                   _vp, _i64, _vp]),
        ("gemm_norm_residual", _st, [_P(gemm_norm_args), _vp]),
        ("gemm_norm_backward_workspace", _i64, [_P(gemm_norm_backward_args)]),
        ("gemm_norm_residual_backward", _st, [_P(gemm_norm_backward_args), _vp])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args

MOE_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 64, 512, 16
NORM_MAX_COLS = 16384

_FLOAT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_GATE_ACT = {"linear": int(Epilogue.LINEAR), "sigmoid": int(Epilogue.SIGMOID)}


# The current device and its current stream's handle, without the objects that
# the public calls build (2.8 us a call).
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _float_type(t: torch.Tensor, name: str) -> int:
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, must be float32, float16 or bfloat16")
    return code


def _device(t: torch.Tensor, name: str) -> int:
    """The index of a tensor's device, which must be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is {_current_device()}")
    return dev


def _rows(t: torch.Tensor, name: str, dev: int, dtype=None, shape=None) -> int:
    """Check a 2-D tensor of contiguous rows on device `dev`; its leading dimension."""
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{name} must be 2-D, has shape {tuple(size)}")
    if t.get_device() != dev:
        _device(t, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, must be {dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, must be {tuple(shape)}")
    rows, cols = size
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows, has strides {t.stride()}")
    if rows <= 1 or cols == 0:
        return cols
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows, strides {t.stride()}")
    return ld


def _vector(t: Optional[torch.Tensor], name: str, dev: int, dtype, n: int) -> Optional[int]:
    if t is None:
        return None
    if t.get_device() != dev:
        _device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, must be {dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous elements, has shape {tuple(t.shape)}")
    return t.data_ptr()


def _streamed(call):
    """Give a call on the current stream a ``stream`` argument (a torch stream or
    a handle): it then runs, and allocates, on that one, and its tensor arguments
    are kept from reuse until the stream has passed the call."""
    @functools.wraps(call)
    def on(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(stream):
            for t in (*args, *kwargs.values()):
                for u in ((t.codes, t.scales) if isinstance(t, Mx4) else (t,)):
                    if isinstance(u, torch.Tensor) and u.is_cuda:
                        u.record_stream(stream)
            return call(*args, **kwargs)
    return on


# ---- MXFP4 ------------------------------------------------------------------------


def gemm_mx4_padded(k: int) -> int:
    return lib.gemm_mx4_padded(k)


class Mx4:
    """An MXFP4 matrix (or a stack of them): uint8 ``codes`` [..., rows, kp/2]
    and ``scales`` [..., rows, kp/32], of rows of ``k`` elements padded to
    kp = ``gemm_mx4_padded(k)``."""

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        kp = gemm_mx4_padded(k)
        for t, name, n in ((codes, "codes", kp // 2), (scales, "scales", kp // 32)):
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous uint8 tensor")
            if t.dim() < 2 or t.shape[-1] != n:
                raise ValueError(f"{name} of rows of {k} elements must end in {n} bytes, has shape "
                                 f"{tuple(t.shape)}")
        if codes.shape[:-1] != scales.shape[:-1]:
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} differ in rows")
        self.codes, self.scales, self.k = codes, scales, k

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]


def _new_mx4(rows: int, k: int, device) -> Mx4:
    kp = -(-k // 256) * 256
    q = object.__new__(Mx4)
    q.codes = torch.empty((rows, kp // 2), dtype=torch.uint8, device=device)
    q.scales = torch.empty((rows, kp // 32), dtype=torch.uint8, device=device)
    q.k = k
    return q


@_streamed
def mx4_quantize(x: torch.Tensor, axis=1):
    """x [R, C] quantised to MXFP4 with blocks along ``axis``: 1 gives R rows of
    C elements, 0 the transposed matrix (C rows of R elements), "both" the pair
    (axis 1, axis 0) from one read of x."""
    if axis not in (0, 1, "both"):
        raise ValueError(f"axis must be 0, 1 or 'both', is {axis!r}")
    code, dev = _float_type(x, "x"), _device(x, "x")
    ld = _rows(x, "x", dev)
    R, C = x.shape
    rows = _new_mx4(R, C, x.device) if axis != 0 else None
    cols = _new_mx4(C, R, x.device) if axis != 1 else None
    _check(lib.gemm_mx4_quantize(
        x.data_ptr(), code, R, C, ld,
        rows and rows.codes.data_ptr(), rows and rows.scales.data_ptr(),
        cols and cols.codes.data_ptr(), cols and cols.scales.data_ptr(), _raw_stream(dev)))
    return (rows, cols) if axis == "both" else cols if rows is None else rows


@_streamed
def mx4_dequantize(q: Mx4, dtype=torch.float32) -> torch.Tensor:
    """The values an MXFP4 matrix stands for."""
    if dtype not in _FLOAT:
        raise TypeError(f"dtype {dtype} must be float32, float16 or bfloat16")
    codes, scales = q.codes, q.scales
    dev = _device(codes, "codes")
    if scales.get_device() != dev:
        _device(scales, "scales")
    lead = codes.shape[:-1]
    out = torch.empty((*lead, q.k), dtype=dtype, device=codes.device)
    _check(lib.gemm_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), lead.numel(), q.k,
                                   out.data_ptr(), _FLOAT[dtype], q.k, _raw_stream(dev)))
    return out


class Mx4Linear:
    """y = act(Q(x) W^T + bias) on MXFP4 operands, and its gradients.

    ``weight``: W [N, K] as an Mx4 of N rows of K elements (what ``forward``
    reads, may be None); ``weight_t``: W quantised along N, an Mx4 of K rows of
    N elements (what the gradient of x reads, may be None). Like a Plan, one
    layer does not run on two streams at once, and its first run of a shape may
    allocate the plan's workspace (so it is not captured into a graph)."""

    def __init__(self, weight: Optional[Mx4], weight_t: Optional[Mx4] = None,
                 activation: str = "linear"):
        if weight is None and weight_t is None:
            raise ValueError("Mx4Linear needs weight or weight_t")
        for w, name in ((weight, "weight"), (weight_t, "weight_t")):
            if w is not None and (w.codes.dim() != 2 or not w.codes.is_cuda or not w.scales.is_cuda):
                raise ValueError(f"{name} must be one MXFP4 matrix on the device")
        if weight is not None and weight_t is not None and (weight_t.rows, weight_t.k) != (
                weight.k, weight.rows):
            raise ValueError(f"weight is {weight.rows} x {weight.k}, weight_t "
                             f"{weight_t.rows} x {weight_t.k}")
        self.weight, self.weight_t = weight, weight_t
        self.N, self.K = ((weight.rows, weight.k) if weight is not None
                          else (weight_t.k, weight_t.rows))
        self.plan = Plan("f4e2m1", la="row", lb="col", lc="row", activation=activation)

    @classmethod
    def from_weight(cls, w: torch.Tensor, backward: bool = False, activation: str = "linear"):
        """Quantise a weight [N, K] for the forward product, and for the
        gradient of x too where ``backward``."""
        if backward:
            return cls(*mx4_quantize(w, "both"), activation=activation)
        return cls(mx4_quantize(w, 1), activation=activation)

    def close(self):
        self.plan.close()

    def _handle(self):
        if self.plan.handle is None:
            raise GemmError(Status.NOT_INITIALIZED, "Mx4Linear: it was closed")
        return self.plan.handle

    @_streamed
    def forward(self, x: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [M, K] (float32, float16 or bfloat16), bias [N] bfloat16 -> [M, N] bfloat16."""
        w = self.weight
        if w is None:
            raise ValueError("forward needs weight, only weight_t was given")
        code, dev = _float_type(x, "x"), _device(x, "x")
        ld = _rows(x, "x", dev)
        M, N, K = x.shape[0], self.N, self.K
        if x.shape[1] != K:
            raise ValueError(f"x has {x.shape[1]} columns, the weight {K}")
        b = _vector(bias, "bias", dev, torch.bfloat16, N)
        need = lib.gemm_mx4_linear_workspace(M, K)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        elif _rows(out, "out", dev, torch.bfloat16, (M, N)) != N:
            raise ValueError("out must be contiguous")
        _check(lib.gemm_mx4_linear(self._handle(), x.data_ptr(), code, ld, w.codes.data_ptr(),
                                   w.scales.data_ptr(), b, out.data_ptr(), M, N, K,
                                   ws.data_ptr() if need else None, need, _raw_stream(dev)))
        return out

    @_streamed
    def backward(self, dy: torch.Tensor, x: Optional[torch.Tensor] = None, need_dx: bool = True,
                 need_dw: bool = True):
        """(dx [M, K], dw [N, K]) in bfloat16 from dy [M, N] and x [M, K] of one
        type; None for one that is not needed."""
        code, dev = _float_type(dy, "dy"), _device(dy, "dy")
        ld = _rows(dy, "dy", dev)
        M, N, K = dy.shape[0], self.N, self.K
        if dy.shape[1] != N:
            raise ValueError(f"dy has {dy.shape[1]} columns, the weight {N} rows")
        if need_dx and self.weight_t is None:
            raise ValueError("the gradient of x needs weight_t")
        ldx = 0
        if need_dw:
            if x is None:
                raise ValueError("the gradient of the weight needs x")
            ldx = _rows(x, "x", dev, dy.dtype, (M, K))
        need = lib.gemm_mx4_linear_backward_workspace(M, N, K)
        ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device) if need_dx else None
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=dy.device) if need_dw else None
        wt = self.weight_t if need_dx else None
        _check(lib.gemm_mx4_linear_backward(
            self._handle(), dy.data_ptr(), ld, x.data_ptr() if need_dw else None, ldx, code,
            wt and wt.codes.data_ptr(), wt and wt.scales.data_ptr(),
            dx.data_ptr() if need_dx else None, dw.data_ptr() if need_dw else None, M, N, K,
            ws.data_ptr(), need, _raw_stream(dev)))
        return dx, dw


# ---- mixture of experts --------------------------------------------------------------


class MoeLayer:
    """A mixture-of-experts layer for up to ``MOE_MAX_TOKENS`` tokens a call.

    ``router`` [E, H] and x are float16 or bfloat16; ``up`` [E, 2 I, H] (the
    gate's rows first) and ``down`` [E, H, I] are tensors of that type, or Mx4
    stacks with bfloat16. Each chosen expert gives down (silu(gate x) * (up x))."""

    def __init__(self, router: torch.Tensor, up, down, top_k: int, renormalize: bool = True):
        code = _float_type(router, "router")
        if router.dim() != 2 or not router.is_cuda or not router.is_contiguous():
            raise ValueError("router must be a contiguous [experts, hidden] device tensor")
        E, H = router.shape
        packed = isinstance(up, Mx4)
        if packed != isinstance(down, Mx4):
            raise TypeError("up and down must both be Mx4 or both be tensors")
        parts = [(up, "up"), (down, "down")]
        if packed:
            shapes = [(*w.codes.shape[:-1], w.k) for w, _ in parts]
            parts = [(t, f"{n} {s}") for w, n in parts for t, s in ((w.codes, "codes"), (w.scales, "scales"))]
        else:
            shapes = [tuple(w.shape) for w, _ in parts]
            for w, name in parts:
                if w.dtype != router.dtype:
                    raise TypeError(f"{name} has dtype {w.dtype}, must be {router.dtype}")
        for t, name in parts:
            if not t.is_cuda or t.device != router.device or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous on the router's device")
        inner = shapes[1][-1]
        if shapes[0] != (E, 2 * inner, H) or shapes[1] != (E, H, inner):
            raise ValueError(f"router {tuple(router.shape)}, up {shapes[0]} and down {shapes[1]} do not "
                             "fit [E, H], [E, 2 I, H] and [E, H, I]")
        self.top_k, self.hidden, self.dtype = top_k, H, router.dtype
        self._keep = (router, up, down)
        wc = (lambda w: (w.codes.data_ptr(), w.scales.data_ptr())) if packed else (
            lambda w: (w.data_ptr(), None))
        self.desc = gemm_moe_desc(H, inner, E, top_k, int(bool(renormalize)), code,
                                  int(Dtype.F4_E2M1) if packed else code, router.data_ptr(),
                                  *wc(up), *wc(down))
        self._ref = ctypes.byref(self.desc)
        need = lib.gemm_moe_workspace(self._ref, MOE_MAX_TOKENS)
        if need < 0:
            _check(lib.gemm_moe_forward(self._ref, None, 0, None, None, 0, None, None, 0, None, 0, None))
        self._bytes, self._state = need, lib.gemm_moe_state_bytes(self._ref)
        self._workspaces = {}

    def _workspace(self, st: int, device) -> torch.Tensor:
        """A workspace whose state is zero: one per stream, kept; a captured
        call gets one of its own, cleared in the graph."""
        capturing = torch.cuda.is_current_stream_capturing()
        ws = None if capturing else self._workspaces.get(st)
        if ws is None:
            ws = torch.empty(self._bytes, dtype=torch.uint8, device=device)
            ws[:self._state].zero_()
            if not capturing:
                self._workspaces[st] = ws
        return ws

    @_streamed
    def __call__(self, x: torch.Tensor, row_mask: Optional[torch.Tensor] = None,
                 return_routing: bool = False, out: Optional[torch.Tensor] = None):
        """x [T, H] -> [T, H]; with ``return_routing`` also the chosen experts
        [T, top_k] int32 and their weights [T, top_k] float32. ``row_mask`` [T]
        (bool or uint8): tokens where it is false are routed nowhere and get 0."""
        dev = _device(x, "x")
        ldx = _rows(x, "x", dev, self.dtype)
        T, H = x.shape
        if H != self.hidden:
            raise ValueError(f"x has {H} columns, the layer {self.hidden}")
        mask = None
        if row_mask is not None:
            if row_mask.dtype == torch.bool:
                row_mask = row_mask.view(torch.uint8)
            mask = _vector(row_mask, "row_mask", dev, torch.uint8, T)
        if out is None:
            out, ldo = torch.empty((T, H), dtype=self.dtype, device=x.device), H
        else:
            ldo = _rows(out, "out", dev, self.dtype, (T, H))
        ids = probs = None
        if return_routing:
            ids = torch.empty((T, self.top_k), dtype=torch.int32, device=x.device)
            probs = torch.empty((T, self.top_k), dtype=torch.float32, device=x.device)
        st = _raw_stream(dev)
        ws = self._workspace(st, x.device)
        _check(lib.gemm_moe_forward(self._ref, x.data_ptr(), ldx, mask, out.data_ptr(), ldo,
                                    ids.data_ptr() if return_routing else None,
                                    probs.data_ptr() if return_routing else None, T,
                                    ws.data_ptr(), self._bytes, st))
        return (out, ids, probs) if return_routing else out


# ---- norms around a block ---------------------------------------------------------------


def _gate_rows(gate, dev, dtype, rows, cols):
    ld = _rows(gate, "gate", dev, dtype)
    g = gate.shape[0]
    if gate.shape[1] != cols or (rows > 0 and (g == 0 or rows % g)):
        raise ValueError(f"gate has shape {tuple(gate.shape)}: its rows must divide {rows} rows of "
                         f"{cols} columns")
    return g, ld


def _act(gate_act: str) -> int:
    act = _GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(_GATE_ACT)}, is {gate_act!r}")
    return act


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


@_streamed
def norm_residual(block, residual, *, w_post=None, gate=None, scale=None, w_next=None,
                  eps: float = 1e-6, gate_act: str = "linear"):
    """out = residual + scale * act(gate) * RMSnorm(block) * w_post and
    next = RMSnorm(out) * w_next, as (out, next, saved).

    ``block`` None: only next = RMSnorm(residual) * w_next, out is residual.
    ``w_post`` None: no norm after the block; ``w_next`` None: next is None.
    ``gate`` [G, H]: one row for every T / G consecutive rows; ``gate_act``
    "linear" or "sigmoid". ``saved`` is what norm_residual_backward takes."""
    code, dev = _float_type(residual, "residual"), _device(residual, "residual")
    ldr = _rows(residual, "residual", dev)
    dt, size, device = residual.dtype, residual.shape, residual.device
    T, H = size
    ldb = _rows(block, "block", dev, dt, size) if block is not None else 0
    g, ldg = _gate_rows(gate, dev, dt, T, H) if gate is not None else (0, 0)
    act = _act(gate_act)
    wp, sc, wn = (_vector(w_post, "w_post", dev, dt, H), _vector(scale, "scale", dev, dt, H),
                  _vector(w_next, "w_next", dev, dt, H))
    saved = torch.empty((2, T), dtype=torch.float32, device=device)
    out = residual if block is None else torch.empty(size, dtype=dt, device=device)
    nxt = torch.empty(size, dtype=dt, device=device) if w_next is not None else None
    p = saved.data_ptr()
    a = gemm_norm_args(code, act, T, H, g, eps, _ptr(block), residual.data_ptr(), _ptr(gate), ldb, ldr,
                       ldg, wp, sc, wn, out.data_ptr() if block is not None else None, _ptr(nxt), H, H,
                       p, p + 4 * T)
    _check(lib.gemm_norm_residual(ctypes.byref(a), _raw_stream(dev)))
    return out, nxt, saved


@_streamed
def norm_residual_backward(d_out, d_next, block, out, saved, *, w_post=None, gate=None, scale=None,
                           w_next=None, gate_act: str = "linear") -> dict:
    """Gradients of norm_residual from those of its results (``d_out`` may be
    None for zero; ``d_next`` is given where w_next is). ``out`` and ``saved``
    are what it returned. Gives d_block, d_residual, d_gate, d_scale, d_w_post
    and d_w_next, None where the input is None."""
    code, dev = _float_type(out, "out"), _device(out, "out")
    ldo = _rows(out, "out", dev)
    dt, size, device = out.dtype, out.shape, out.device
    T, H = size
    if (d_next is None) != (w_next is None):
        raise ValueError("d_next and w_next go together")
    if saved.dtype != torch.float32 or saved.shape != (2, T) or not saved.is_contiguous():
        raise ValueError("saved must be what norm_residual returned for these rows")
    if saved.get_device() != dev:
        _device(saved, "saved")
    ldb = _rows(block, "block", dev, dt, size) if block is not None else 0
    lddo = _rows(d_out, "d_out", dev, dt, size) if d_out is not None else 0
    lddn = _rows(d_next, "d_next", dev, dt, size) if d_next is not None else 0
    g, ldg = _gate_rows(gate, dev, dt, T, H) if gate is not None else (0, 0)
    act = _act(gate_act)
    wp, sc, wn = (_vector(w_post, "w_post", dev, dt, H), _vector(scale, "scale", dev, dt, H),
                  _vector(w_next, "w_next", dev, dt, H))
    p = saved.data_ptr()
    a = gemm_norm_backward_args(code, act, T, H, g, _ptr(d_out), _ptr(d_next), _ptr(block), out.data_ptr(),
                                _ptr(gate), lddo, lddn, ldb, ldo, ldg, wp, sc, wn, p, p + 4 * T)
    ref = ctypes.byref(a)
    need = lib.gemm_norm_backward_workspace(ref)
    if need < 0:
        _check(lib.gemm_norm_residual_backward(ref, _raw_stream(dev)))
    d_block = torch.empty(size, dtype=dt, device=device) if block is not None else None
    d_residual = torch.empty(size, dtype=dt, device=device)
    d_gate = torch.empty((g, H), dtype=dt, device=device) if gate is not None else None
    d_scale = torch.empty(H, dtype=dt, device=device) if scale is not None else None
    d_w_post = torch.empty(H, dtype=dt, device=device) if w_post is not None else None
    d_w_next = torch.empty(H, dtype=dt, device=device) if w_next is not None else None
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    a.d_block, a.d_residual, a.ld_d_block, a.ld_d_residual = _ptr(d_block), d_residual.data_ptr(), H, H
    a.d_gate, a.d_scale, a.d_w_post, a.d_w_next = _ptr(d_gate), _ptr(d_scale), _ptr(d_w_post), _ptr(d_w_next)
    a.workspace, a.workspace_bytes = ws.data_ptr(), need
    _check(lib.gemm_norm_residual_backward(ref, _raw_stream(dev)))
    return {"d_block": d_block, "d_residual": d_residual, "d_gate": d_gate, "d_scale": d_scale,
            "d_w_post": d_w_post, "d_w_next": d_w_next}
