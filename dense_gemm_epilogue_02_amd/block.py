"""Binding of the feed-forward block's operators (``include/gemm_block.h``):
MXFP4 operands and the linear layer on them, the mixture-of-experts layer for a
few tokens, and the norms around a block.

Argument marshalling only, most of it in the extension ``_block`` (a call in
ctypes takes as long as its kernels for a few tokens). Tensors are 2-D device
tensors whose rows are contiguous (any distance between rows). Results and
workspaces are allocated by torch on the stream that the kernels are enqueued on
(torch's current one, unless ``stream`` is given). Nothing here takes part in
autograd: the backward passes are calls of their own.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import Dtype, Epilogue, GemmError, Plan, Status, _check, lib


class _NotLoaded:
    """Stands for an extension that does not load: its first use says so. The
    GEMMs need the library alone, so importing the package does not fail."""

    def __init__(self, error: ImportError, name: str = "_block"):
        self.__dict__.update(error=error, name=name)

    def __getattr__(self, name):
        raise ImportError(f"the extension {self.name} is not built or does not load; run `python -c 'import __graft_entry__ "
                          "as g; g.build()'` from the repository root") from self.error


try:
    from . import _block
    _block.set_check(_check)
except ImportError as _error:
    _block = _NotLoaded(_error)

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


def _float_type(t: torch.Tensor, name: str) -> int:
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, must be float32, float16 or bfloat16")
    return code


def _on(stream, call, *args, keep=()):
    """A call on another stream (a torch stream or a handle): it runs, and
    allocates, there, and its tensor arguments, and the tensors in ``keep`` that
    it reads besides (a layer's weights), are kept from reuse until the stream
    has passed it."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        for t in (*args, *keep):
            for u in ((t.codes, t.scales) if isinstance(t, Mx4) else (t,)):
                if isinstance(u, torch.Tensor) and u.is_cuda:
                    u.record_stream(stream)
        return call(*args)


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


def _mx4(codes, scales, k: int) -> Mx4:
    q = object.__new__(Mx4)
    q.codes, q.scales, q.k = codes, scales, k
    return q


def mx4_quantize(x: torch.Tensor, axis=1, stream=None):
    """x [R, C] quantised to MXFP4 with blocks along ``axis``: 1 gives R rows of
    C elements, 0 the transposed matrix (C rows of R elements), "both" the pair
    (axis 1, axis 0) from one read of x."""
    if axis not in (0, 1, "both"):
        raise ValueError(f"axis must be 0, 1 or 'both', is {axis!r}")
    if stream is not None:
        return _on(stream, mx4_quantize, x, axis)
    rc, rs, cc, cs = _block.quantize(x, axis != 0, axis != 1)
    if axis == 1:
        return _mx4(rc, rs, x.shape[1])
    cols = _mx4(cc, cs, x.shape[0])
    return cols if axis == 0 else (_mx4(rc, rs, x.shape[1]), cols)


def mx4_dequantize(q: Mx4, dtype=torch.float32, stream=None) -> torch.Tensor:
    """The values an MXFP4 matrix stands for."""
    if stream is not None:
        return _on(stream, mx4_dequantize, q, dtype)
    return _block.dequantize(q.codes, q.scales, q.k, dtype)


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
            if w is not None and (w.codes.dim() != 2 or not w.codes.is_cuda or w.scales.device != w.codes.device):
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

    def forward(self, x: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x [M, K] (float32, float16 or bfloat16), bias [N] bfloat16 -> [M, N] bfloat16."""
        if stream is not None:
            return _on(stream, self.forward, x, bias, out, keep=(self.weight,))
        w = self.weight
        if w is None:
            raise ValueError("forward needs weight, only weight_t was given")
        return _block.linear(self._handle(), x, w.codes, w.scales, self.N, self.K, bias, out)

    def backward(self, dy: torch.Tensor, x: Optional[torch.Tensor] = None, need_dx: bool = True,
                 need_dw: bool = True, stream=None):
        """(dx [M, K], dw [N, K]) in bfloat16 from dy [M, N] and x [M, K] of one
        type; None for one that is not needed."""
        if stream is not None:
            return _on(stream, self.backward, dy, x, need_dx, need_dw, keep=(self.weight_t,))
        wt = self.weight_t
        if need_dx and wt is None:
            raise ValueError("the gradient of x needs weight_t")
        if need_dw and x is None:
            raise ValueError("the gradient of the weight needs x")
        return _block.linear_backward(self._handle(), dy, x, wt and wt.codes, wt and wt.scales, self.N, self.K,
                                      bool(need_dx), bool(need_dw))


# ---- mixture of experts --------------------------------------------------------------


class MoeLayer:
    """A mixture-of-experts layer for up to ``MOE_MAX_TOKENS`` tokens a call (more
    are calls of their own).

    ``router`` [E, H] and x are float16 or bfloat16; ``up`` [E, 2 I, H] (the
    gate's rows first) and ``down`` [E, H, I] are tensors of that type, or Mx4
    stacks with bfloat16. Each chosen expert gives down (silu(gate x) * (up x)),
    whose bracket is not rounded to the type and may pass its range."""

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
        self._ref, self._at = ctypes.byref(self.desc), ctypes.addressof(self.desc)
        need = lib.gemm_moe_workspace(self._ref, MOE_MAX_TOKENS)
        if need < 0:
            _check(lib.gemm_moe_forward(self._ref, None, 0, None, None, 0, None, None, 0, None, 0, None))
        self._bytes, self._state = need, lib.gemm_moe_state_bytes(self._ref)
        self._workspaces = {}

    def _workspace(self, x: torch.Tensor) -> torch.Tensor:
        """A workspace whose state is zero: one per stream, kept; a captured
        call gets one of its own, cleared in the graph."""
        if not x.is_cuda:
            raise ValueError("x must be a device tensor")
        capturing = torch.cuda.is_current_stream_capturing()
        st = torch._C._cuda_getCurrentRawStream(x.get_device())
        ws = None if capturing else self._workspaces.get(st)
        if ws is None:
            ws = torch.empty(self._bytes, dtype=torch.uint8, device=x.device)
            ws[:self._state].zero_()
            if not capturing:
                self._workspaces[st] = ws
        return ws

    def __call__(self, x: torch.Tensor, row_mask: Optional[torch.Tensor] = None,
                 return_routing: bool = False, out: Optional[torch.Tensor] = None, stream=None):
        """x [T, H] -> [T, H]; with ``return_routing`` also the chosen experts
        [T, top_k] int32 and their weights [T, top_k] float32. ``row_mask`` [T]
        (bool or uint8): tokens where it is false are routed nowhere and get 0."""
        if stream is not None:
            return _on(stream, self.__call__, x, row_mask, return_routing, out, keep=self._keep)
        r = _block.moe(self._at, x, row_mask, out, bool(return_routing), self._workspace(x), self._keep[0])
        return r if return_routing else r[0]


# ---- norms around a block ---------------------------------------------------------------


def _act(gate_act: str) -> int:
    act = _GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(_GATE_ACT)}, is {gate_act!r}")
    return act


def norm_residual(block, residual, *, w_post=None, gate=None, scale=None, w_next=None,
                  eps: float = 1e-6, gate_act: str = "linear", stream=None):
    """out = residual + scale * act(gate) * RMSnorm(block) * w_post and
    next = RMSnorm(out) * w_next, as (out, next, saved).

    ``block`` None: only next = RMSnorm(residual) * w_next, out is residual.
    ``w_post`` None: no norm after the block; ``w_next`` None: next is None.
    ``gate`` [G, H]: one row for every T / G consecutive rows; ``gate_act``
    "linear" or "sigmoid". ``saved`` is what norm_residual_backward takes."""
    args = (block, residual, w_post, gate, scale, w_next, eps, _act(gate_act))
    return _block.norm(*args) if stream is None else _on(stream, _block.norm, *args)


def norm_residual_backward(d_out, d_next, block, out, saved, *, w_post=None, gate=None, scale=None,
                           w_next=None, gate_act: str = "linear", stream=None) -> dict:
    """Gradients of norm_residual from those of its results (``d_out`` may be
    None for zero; ``d_next`` is given where w_next is). ``out`` and ``saved``
    are what it returned. Gives d_block, d_residual, d_gate, d_scale, d_w_post
    and d_w_next, None where the input is None."""
    args = (d_out, d_next, block, out, saved, w_post, gate, scale, w_next, _act(gate_act))
    d = _block.norm_backward(*args) if stream is None else _on(stream, _block.norm_backward, *args)
    return dict(zip(_GRADIENTS, d))


_GRADIENTS = ("d_block", "d_residual", "d_gate", "d_scale", "d_w_post", "d_w_next")
