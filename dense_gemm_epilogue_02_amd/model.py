"""Binding of the operators around a language model's products
(``include/gemm_model.h``): losses of the output head whose logits are not
kept, and tokens sorted by expert.

Argument marshalling only, most of it in the extension ``_model``. Matrices are
2-D device tensors whose rows are contiguous (any distance between rows), all
other tensors are contiguous. Results and workspaces are allocated by torch on
the stream that the kernels are enqueued on (torch's current one, unless
``stream`` is given). Nothing here takes part in autograd: the backward passes
are calls of their own.
"""
from __future__ import annotations

import ctypes
from typing import List, Optional, Tuple

import torch

from . import _check, lib
from .block import _NotLoaded, _on

try:
    from . import _model
    _model.set_check(_check)
except ImportError as _error:
    _model = _NotLoaded(_error, "_model")

_i32, _i64, _f32, _vp, _st = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int


class gemm_head_args(ctypes.Structure):
    _fields_ = [("type", _st), ("tokens", _i64), ("hidden", _i64), ("vocab", _i64), ("x", _vp), ("ldx", _i64), ("w", _vp),
                ("scale", _f32), ("z_loss", _f32), ("targets", _vp), ("target_bits", _i32), ("ignore_index", _i64),
                ("teacher_ids", _vp), ("teacher_logits", _vp), ("ld_teacher", _i64), ("teacher_type", _st),
                ("entries", _i32), ("temperature", _f32)]


class gemm_head_saved(ctypes.Structure):
    _fields_ = [("lse", _vp), ("picked", _vp), ("ids", _vp), ("weights", _vp), ("mass", _vp)]


_A, _S = ctypes.POINTER(gemm_head_args), ctypes.POINTER(gemm_head_saved)
for _name, _res, _args in (
        ("gemm_head_workspace", _i64, [_A, _i32]),
        ("gemm_head_loss", _st, [_A, _vp, _S, _vp, _i64, _vp]),
        ("gemm_head_backward", _st, [_A, _vp, _S, _vp, _vp, _vp, _i64, _vp]),
        ("gemm_expert_sort_workspace", _i64, [_i64, _i32, _i32]),
        ("gemm_expert_sort", _st, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp]),
        ("gemm_expert_gather", _st, [_st, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp]),
        ("gemm_expert_combine", _st, [_st, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp]),
        ("gemm_expert_combine_backward", _st, [_st, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _i32,
                                               _vp, _vp, _vp])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args

HEAD_MAX_ENTRIES, EXPERT_MAX_EXPERTS = 256, 1024

# ---- losses of the output head -------------------------------------------------------


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                         scale: float = 1.0, z_loss: float = 0.0, stream=None) -> Tuple[torch.Tensor, tuple]:
    """The cross entropy of logits scale * x W^T, which are never written, for
    each token: (loss [T] float32, saved).

    ``x`` [T, H] and ``w`` [V, H] (contiguous) are float16 or bfloat16,
    ``targets`` [T] int32 or int64. loss = lse - logit[target] + z_loss * lse^2
    with lse the logarithm of the logits' summed exponentials; 0 where the target
    is ``ignore_index``, NaN where another one lies outside the vocabulary.
    ``saved`` is what linear_cross_entropy_backward takes."""
    args = (x, w, targets, ignore_index, scale, z_loss)
    loss, *saved = _model.cross_entropy(*args) if stream is None else _on(stream, _model.cross_entropy, *args)
    return loss, tuple(saved)


def _kept(saved, n: int, whose: str) -> tuple:
    if not isinstance(saved, tuple) or len(saved) != n:
        raise ValueError(f"saved must be what {whose} returned for these tokens")
    return saved


def linear_cross_entropy_backward(d_loss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                                  saved: tuple, *, ignore_index: int = -100, scale: float = 1.0, z_loss: float = 0.0,
                                  need_dx: bool = True, need_dw: bool = True, stream=None) -> tuple:
    """(dx [T, H], dw [V, H]) of the sum of d_loss * loss, in x's type; None for
    one that is not needed. ``d_loss`` [T] float32; the other arguments are the
    forward pass's. Tokens without a label or whose d_loss is 0 take no work,
    and what lies in their rows of x reaches nothing."""
    args = (d_loss, x, w, *_kept(saved, 2, "linear_cross_entropy"), targets, ignore_index, scale, z_loss, bool(need_dx),
            bool(need_dw))
    call = _model.cross_entropy_backward
    return call(*args) if stream is None else _on(stream, call, *args)


def linear_distillation(x: torch.Tensor, w: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                        temperature: float = 1.0, scale: float = 1.0, stream=None) -> Tuple[torch.Tensor, tuple]:
    """temperature^2 times the divergence of softmax(scale * x W^T /
    temperature) from a teacher's distribution, for each token: (loss [T]
    float32, saved).

    The teacher's distribution is the softmax of ``teacher_logits`` [T, K]
    (float32, float16 or bfloat16) / temperature over the entries
    ``teacher_ids`` [T, K] int32 of the vocabulary (K <= HEAD_MAX_ENTRIES).
    Entries with a negative id do not exist, entries of one id count as one of
    their summed weight, a token without entries has loss 0. An id past the
    vocabulary gives NaN."""
    args = (x, w, teacher_ids, teacher_logits, temperature, scale)
    loss, *saved = _model.distillation(*args) if stream is None else _on(stream, _model.distillation, *args)
    return loss, tuple(saved)


def linear_distillation_backward(d_loss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, saved: tuple, *,
                                 temperature: float = 1.0, scale: float = 1.0, need_dx: bool = True,
                                 need_dw: bool = True, stream=None) -> tuple:
    """(dx [T, H], dw [V, H]) of the sum of d_loss * loss, in x's type; None for
    one that is not needed. ``saved`` is what linear_distillation returned, the
    other arguments are its own."""
    args = (d_loss, x, w, *_kept(saved, 5, "linear_distillation"), temperature, scale, bool(need_dx), bool(need_dw))
    call = _model.distillation_backward
    return call(*args) if stream is None else _on(stream, call, *args)


# ---- tokens by expert ------------------------------------------------------------------


class ExpertOrder:
    """Slots (a token and one of its choices) in the order of their experts:
    ``offsets`` [E + 1] int32, expert e has rows offsets[e] .. offsets[e + 1);
    ``row_of`` [T, top_k] int32, each slot's row, -1 for one routed nowhere."""

    __slots__ = ("offsets", "row_of")

    def __init__(self, offsets: torch.Tensor, row_of: torch.Tensor):
        self.offsets, self.row_of = offsets, row_of

    @property
    def experts(self) -> int:
        return self.offsets.shape[0] - 1

    @property
    def tokens(self) -> int:
        return self.row_of.shape[0]

    @property
    def top_k(self) -> int:
        return self.row_of.shape[1]

    def bounds(self) -> List[int]:
        """``offsets`` on the host, as a grouped GEMM's sizes are given; waits
        for the sort."""
        return self.offsets.tolist()


def expert_sort(ids: torch.Tensor, experts: int, stream=None) -> ExpertOrder:
    """The order of the slots ids [T, top_k] (int32 or int64) by expert, those of
    one expert by token and choice. Ids outside [0, experts) are routed nowhere;
    a token may choose an expert twice."""
    args = (ids, experts)
    return ExpertOrder(*(_model.expert_sort(*args) if stream is None else _on(stream, _model.expert_sort, *args)))


def expert_gather(x: torch.Tensor, order: ExpertOrder, stream=None) -> torch.Tensor:
    """x [T, H] to rows [T * top_k, H] in the order of their experts; rows behind
    the last expert's are 0. float32, float16 or bfloat16."""
    args = (x, order.offsets, order.row_of)
    return _model.expert_gather(*args) if stream is None else _on(stream, _model.expert_gather, *args)


def expert_gather_backward(d_rows: torch.Tensor, order: ExpertOrder, stream=None) -> torch.Tensor:
    """The gradient of expert_gather's x: the sum of each token's rows of d_rows."""
    return expert_combine(d_rows, order, None, stream)


def expert_combine(rows: torch.Tensor, order: ExpertOrder, weights: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """rows [T * top_k, H] to out [T, H]: the sum of each token's rows times
    ``weights`` [T, top_k] float32 (None: 1), in fp32 and rounded once."""
    args = (rows, order.offsets, order.row_of, weights)
    return _model.expert_combine(*args) if stream is None else _on(stream, _model.expert_combine, *args)


def expert_combine_backward(d_out: torch.Tensor, rows: torch.Tensor, order: ExpertOrder,
                            weights: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """(d_rows [T * top_k, H], d_weights [T, top_k] float32) of expert_combine
    from d_out [T, H] and its rows; d_weights is None where weights is."""
    args = (d_out, rows, order.offsets, order.row_of, weights)
    call = _model.expert_combine_backward
    return call(*args) if stream is None else _on(stream, call, *args)
