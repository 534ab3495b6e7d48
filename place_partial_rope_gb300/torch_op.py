"""PyTorch operator and autograd for the in-place partial rotary embedding.

The user-facing API described by "CANN ops-transformer
inplace_partial_rotary_mul" (sections 函数原型与参数说明, 自动微分说明 and
图模式调用), on top of the C ABI:

    inplace_partial_rotary_mul(x, r1, r2, *, rotary_mode="interleave",
                               partial_slice=None) -> None

* Operator schema (namespace ``place_partial_rope``):
  ``inplace_partial_rotary_mul(Tensor(a!) x, Tensor r1, Tensor r2, *,
  str rotary_mode='interleave', int[2] partial_slice=[0, 0]) -> ()`` and
  ``inplace_partial_rotary_mul_backward(Tensor(a!) grad, Tensor r1,
  Tensor r2, *, str rotary_mode='interleave', int[2] partial_slice=[0, 0]) -> ()``.
  Both have a CUDA kernel (the library) and a Meta kernel (shape checks
  only, for fake tensors and tracing).  There is no CPU kernel: CPU tensors
  fail in the dispatcher.
* ``partial_slice=None`` means [0, 0], an empty slice (a no-op).
* ``rotary_mode``: "interleave" (the page's only mode: pairs (2i, 2i+1)) or
  "half" (half-split rotate_half: pairs (i, i + L/2)); anything else raises.
* When ``x.requires_grad`` and grad mode is on, the call goes through
  ``InplacePartialRotaryMulFn``: the forward marks x dirty and saves r1 and
  r2; the backward applies the transposed rotation to the incoming
  gradient and returns no gradient for r1 and r2.  As with any in-place op,
  x must not be a leaf that requires grad (use ``y = x * 1.0`` first).
* The backward writes into its own contiguous copy of the incoming gradient,
  so a gradient that autograd also hands to someone else (``retain_grad``,
  an expanded gradient of a sum) is never changed.

Rotary positions with several axes, with the same rules (in place, Meta kernel,
autograd; the positions get no gradient):

    inplace_axes_rotary_mul(x, positions, sections, *, rotary_mode="interleave",
                            partial_slice=None, base=10000.0, order="blocked",
                            spectrum="shared") -> None

Norm and rotation of query and key rows in one pass, out of place, with gradients of
the rows and of the weights (cos and sin get none; no second gradients):

    norm_rotary(q, k, q_weight, k_weight, cos, sin, *, rotary_mode="interleave",
                partial_slice=None, norm_slice=None, eps=1e-6) -> (q_out, k_out)
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import binding

NAMESPACE = "place_partial_rope"
_FWD = "inplace_partial_rotary_mul"
_BWD = "inplace_partial_rotary_mul_backward"
_AXES_FWD = "inplace_axes_rotary_mul"
_AXES_BWD = "inplace_axes_rotary_mul_backward"
_NORM_FWD = "norm_rotary"
_NORM_BWD = "norm_rotary_backward"
_MODES = ("interleave", "half")

_lib = None


def _check(x: torch.Tensor, rotary_mode: str, partial_slice: Sequence[int]) -> None:
    """The compile-time checks of the page's Meta implementation."""
    if x.dim() != 4:
        raise ValueError(f"inplace_partial_rotary_mul: x must be 4-D (B, S, N, D), got {x.dim()}-D")
    if rotary_mode not in _MODES:
        raise ValueError(f"inplace_partial_rotary_mul: rotary_mode must be 'interleave' or "
                         f"'half', got {rotary_mode!r}")
    if len(partial_slice) != 2:
        raise ValueError(f"inplace_partial_rotary_mul: partial_slice must hold 2 integers, "
                         f"got {len(partial_slice)}")


def _cuda_fwd(x, r1, r2, rotary_mode="interleave", partial_slice=(0, 0)):
    _check(x, rotary_mode, partial_slice)
    binding.rope_partial_inplace_fwd_mode(x, r1, r2, int(partial_slice[0]), int(partial_slice[1]),
                                          rotary_mode)


def _cuda_bwd(grad, r1, r2, rotary_mode="interleave", partial_slice=(0, 0)):
    _check(grad, rotary_mode, partial_slice)
    binding.rope_partial_inplace_bwd_mode(grad, r1, r2, int(partial_slice[0]),
                                          int(partial_slice[1]), rotary_mode)


def _meta(x, r1, r2, rotary_mode="interleave", partial_slice=(0, 0)):
    _check(x, rotary_mode, partial_slice)
    return None


def _check_axes(x, positions, sections, rotary_mode, partial_slice, order, spectrum) -> None:
    if x.dim() != 4:
        raise ValueError(f"inplace_axes_rotary_mul: x must be 4-D (B, S, N, D), got {x.dim()}-D")
    if positions.dim() != 3 or positions.shape[0] != len(sections):
        raise ValueError("inplace_axes_rotary_mul: positions must be 3-D (axes, B|1, S|1) with one "
                         "section per axis")
    if rotary_mode not in _MODES:
        raise ValueError(f"inplace_axes_rotary_mul: rotary_mode must be 'interleave' or 'half', "
                         f"got {rotary_mode!r}")
    if len(partial_slice) != 2:
        raise ValueError(f"inplace_axes_rotary_mul: partial_slice must hold 2 integers, "
                         f"got {len(partial_slice)}")
    if order not in binding.ORDER_CODE or spectrum not in binding.SPECTRUM_CODE:
        raise ValueError(f"inplace_axes_rotary_mul: order {order!r} or spectrum {spectrum!r} is unknown")


def _axes_impl(fn):
    def call(x, positions, sections, rotary_mode="interleave", partial_slice=(0, 0), base=10000.0,
             order="blocked", spectrum="shared"):
        _check_axes(x, positions, sections, rotary_mode, partial_slice, order, spectrum)
        fn(x, positions, sections, int(partial_slice[0]), int(partial_slice[1]), base, rotary_mode, order,
           spectrum)
    return call


def _axes_meta(x, positions, sections, rotary_mode="interleave", partial_slice=(0, 0), base=10000.0,
               order="blocked", spectrum="shared"):
    _check_axes(x, positions, sections, rotary_mode, partial_slice, order, spectrum)
    return None


def _check_norm(q, k, rotary_mode, partial_slice, norm_slice) -> None:
    for x, what in ((q, "q"), (k, "k")):
        if x is not None and x.dim() != 4:
            raise ValueError(f"norm_rotary: {what} must be 4-D (B, S, N, D), got {x.dim()}-D")
    if k is not None and (k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]):
        raise ValueError("norm_rotary: q and k must share B, S and D")
    if rotary_mode not in _MODES:
        raise ValueError(f"norm_rotary: rotary_mode must be 'interleave' or 'half', got {rotary_mode!r}")
    if len(partial_slice) != 2 or len(norm_slice) != 2:
        raise ValueError("norm_rotary: partial_slice and norm_slice must hold 2 integers each")


def _rows(x):
    """x, or a copy whose last dim is contiguous."""
    return x if x is None or x.stride(-1) == 1 or x.shape[-1] <= 1 else x.contiguous()


def _like(x, shape=None, dtype=None):
    """An uninitialised contiguous tensor of x's shape (or another); of nothing for None."""
    if x is None:
        return torch.empty(0)
    return torch.empty(x.shape if shape is None else shape, dtype=dtype or x.dtype, device=x.device)


def _norm_outputs(q, k, keep_rstd):
    return (_like(q), _like(k), *(_like(x if keep_rstd else None, None if x is None else x.shape[:3], torch.float32)
                                  for x in (q, k)))


def _norm_grads(q, k, q_weight, k_weight, weight_grads):
    return (_like(q), _like(k), *(_like(w if wanted else None, None, torch.float32)
                                  for w, wanted in zip((q_weight, k_weight), weight_grads)))


def _norm_cuda(q, k, q_weight, k_weight, cos, sin, rotary_mode="interleave", partial_slice=(0, 0),
               norm_slice=(0, 0), eps=1e-6, keep_rstd=True):
    _check_norm(q, k, rotary_mode, partial_slice, norm_slice)
    q, k = _rows(q), _rows(k)
    got = _norm_outputs(q, k, keep_rstd)
    binding.rope_partial_norm_fwd(q, k, q_weight, k_weight, cos, sin, *partial_slice, eps=eps, norm=tuple(norm_slice),
                                  mode=rotary_mode, q_out=got[0], k_out=None if k is None else got[1],
                                  q_rstd=got[2] if keep_rstd else None,
                                  k_rstd=got[3] if keep_rstd and k is not None else None)
    return got


def _norm_cuda_bwd(dq, dk, q, k, q_weight, k_weight, q_rstd, k_rstd, cos, sin, rotary_mode="interleave",
                   partial_slice=(0, 0), norm_slice=(0, 0), weight_grads=(True, True)):
    _check_norm(q, k, rotary_mode, partial_slice, norm_slice)
    q, k = _rows(q), _rows(k)
    got = _norm_grads(q, k, q_weight, k_weight, weight_grads)
    binding.rope_partial_norm_bwd(_rows(dq), _rows(dk), q, k, q_weight, k_weight, q_rstd, k_rstd, cos, sin,
                                  *partial_slice, norm=tuple(norm_slice), mode=rotary_mode, dq_out=got[0],
                                  dk_out=None if k is None else got[1],
                                  dq_weight=got[2] if q_weight is not None and weight_grads[0] else None,
                                  dk_weight=got[3] if k_weight is not None and weight_grads[1] else None)
    return got


def _norm_meta(q, k, q_weight, k_weight, cos, sin, rotary_mode="interleave", partial_slice=(0, 0),
               norm_slice=(0, 0), eps=1e-6, keep_rstd=True):
    _check_norm(q, k, rotary_mode, partial_slice, norm_slice)
    return _norm_outputs(q, k, keep_rstd)


def _norm_meta_bwd(dq, dk, q, k, q_weight, k_weight, q_rstd, k_rstd, cos, sin, rotary_mode="interleave",
                   partial_slice=(0, 0), norm_slice=(0, 0), weight_grads=(True, True)):
    return _norm_grads(q, k, q_weight, k_weight, weight_grads)


def register() -> None:
    """Define the operators once per process (idempotent)."""
    global _lib
    if _lib is not None:
        return
    lib = torch.library.Library(NAMESPACE, "DEF")
    lib.define(f"{_FWD}(Tensor(a!) x, Tensor r1, Tensor r2, *, str rotary_mode='interleave', "
               "int[2] partial_slice=[0, 0]) -> ()")
    lib.define(f"{_BWD}(Tensor(a!) grad, Tensor r1, Tensor r2, *, str rotary_mode='interleave', "
               "int[2] partial_slice=[0, 0]) -> ()")
    lib.impl(_FWD, _cuda_fwd, "CUDA")
    lib.impl(_BWD, _cuda_bwd, "CUDA")
    lib.impl(_FWD, _meta, "Meta")
    lib.impl(_BWD, _meta, "Meta")
    for name, arg, fn in ((_AXES_FWD, "x", binding.rope_partial_inplace_fwd_axes),
                          (_AXES_BWD, "grad", binding.rope_partial_inplace_bwd_axes)):
        lib.define(f"{name}(Tensor(a!) {arg}, Tensor positions, int[] sections, *, "
                   "str rotary_mode='interleave', int[2] partial_slice=[0, 0], float base=10000.0, "
                   "str order='blocked', str spectrum='shared') -> ()")
        lib.impl(name, _axes_impl(fn), "CUDA")
        lib.impl(name, _axes_meta, "Meta")
    rest = "*, str rotary_mode='interleave', int[2] partial_slice=[0, 0], int[2] norm_slice=[0, 0]"
    lib.define(f"{_NORM_FWD}(Tensor q, Tensor? k, Tensor? q_weight, Tensor? k_weight, Tensor? cos, Tensor? sin, "
               f"{rest}, float eps=1e-06, bool keep_rstd=True) -> (Tensor, Tensor, Tensor, Tensor)")
    lib.define(f"{_NORM_BWD}(Tensor dq, Tensor? dk, Tensor q, Tensor? k, Tensor? q_weight, Tensor? k_weight, "
               f"Tensor q_rstd, Tensor? k_rstd, Tensor? cos, Tensor? sin, {rest}, "
               "bool[2] weight_grads=[True, True]) -> (Tensor, Tensor, Tensor, Tensor)")
    lib.impl(_NORM_FWD, _norm_cuda, "CUDA")
    lib.impl(_NORM_FWD, _norm_meta, "Meta")
    lib.impl(_NORM_BWD, _norm_cuda_bwd, "CUDA")
    lib.impl(_NORM_BWD, _norm_meta_bwd, "Meta")
    _lib = lib


def _op(name: str, back: bool):
    """The operator of that name, or the one of its backward."""
    return getattr(getattr(torch.ops, NAMESPACE), name + "_backward" if back else name)


class InplacePartialRotaryMulFn(torch.autograd.Function):
    """Autograd for the in-place rotation, or (``back``) its transpose, which is
    its gradient as it is the transpose's: r1 and r2 get no gradient."""

    @staticmethod
    def forward(ctx, x, r1, r2, rotary_mode, partial_slice, back=False):
        _op(_FWD, back)(x, r1, r2, rotary_mode=rotary_mode, partial_slice=list(partial_slice))
        ctx.mark_dirty(x)
        ctx.save_for_backward(r1, r2)
        ctx.rotary_mode = rotary_mode
        ctx.partial_slice = list(partial_slice)
        ctx.back = back
        return x

    @staticmethod
    def backward(ctx, grad):
        r1, r2 = ctx.saved_tensors
        g = grad.clone(memory_format=torch.contiguous_format)
        if torch.is_grad_enabled():  # a graph of the gradient is wanted
            g = InplacePartialRotaryMulFn.apply(g, r1, r2, ctx.rotary_mode, ctx.partial_slice, not ctx.back)
        else:
            _op(_FWD, not ctx.back)(g, r1, r2, rotary_mode=ctx.rotary_mode, partial_slice=ctx.partial_slice)
        return g, None, None, None, None, None


def inplace_partial_rotary_mul(x: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor, *,
                               rotary_mode: str = "interleave",
                               partial_slice: Optional[Sequence[int]] = None) -> None:
    """Rotate ``x[..., start:end]`` in place (``partial_slice = [start, end]``,
    default empty).  Returns None; x holds the result."""
    register()
    ps = [0, 0] if partial_slice is None else [int(v) for v in partial_slice]
    _check(x, rotary_mode, ps)
    if x.requires_grad and torch.is_grad_enabled():
        InplacePartialRotaryMulFn.apply(x, r1, r2, rotary_mode, ps)
    else:
        getattr(torch.ops, NAMESPACE).inplace_partial_rotary_mul(
            x, r1, r2, rotary_mode=rotary_mode, partial_slice=ps)
    return None


class InplaceAxesRotaryMulFn(torch.autograd.Function):
    """Autograd for the rotation with several axes, or (``back``) its transpose:
    the positions get no gradient."""

    @staticmethod
    def forward(ctx, x, positions, sections, kwargs, back=False):
        _op(_AXES_FWD, back)(x, positions, sections, **kwargs)
        ctx.mark_dirty(x)
        ctx.save_for_backward(positions)
        ctx.sections, ctx.kwargs, ctx.back = sections, kwargs, back
        return x

    @staticmethod
    def backward(ctx, grad):
        (positions,) = ctx.saved_tensors
        g = grad.clone(memory_format=torch.contiguous_format)
        if torch.is_grad_enabled():
            g = InplaceAxesRotaryMulFn.apply(g, positions, ctx.sections, ctx.kwargs, not ctx.back)
        else:
            _op(_AXES_FWD, not ctx.back)(g, positions, ctx.sections, **ctx.kwargs)
        return g, None, None, None, None


def inplace_axes_rotary_mul(x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int], *,
                            rotary_mode: str = "interleave",
                            partial_slice: Optional[Sequence[int]] = None, base: float = 10000.0,
                            order: str = "blocked", spectrum: str = "shared") -> None:
    """Rotate ``x[..., start:end]`` in place by positions on several axes
    (int32, (axes, B|1, S|1)), ``sections[a]`` of the slice's pairs each; see
    ``binding.rope_partial_inplace_fwd_axes``.  Returns None; x holds the result."""
    register()
    ps = [0, 0] if partial_slice is None else [int(v) for v in partial_slice]
    sections = [int(v) for v in sections]
    _check_axes(x, positions, sections, rotary_mode, ps, order, spectrum)
    kwargs = dict(rotary_mode=rotary_mode, partial_slice=ps, base=float(base), order=order, spectrum=spectrum)
    if x.requires_grad and torch.is_grad_enabled():
        InplaceAxesRotaryMulFn.apply(x, positions, sections, kwargs)
    else:
        getattr(torch.ops, NAMESPACE).inplace_axes_rotary_mul(x, positions, sections, **kwargs)
    return None


class NormRotaryFn(torch.autograd.Function):
    """Autograd for the norm and rotation; cos and sin get no gradient."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, kwargs, eps):
        q_out, k_out, q_rstd, k_rstd = _op(_NORM_FWD, False)(q, k, q_weight, k_weight, cos, sin, **kwargs, eps=eps)
        ctx.save_for_backward(q, k, q_weight, k_weight, q_rstd, k_rstd if k is not None else None, cos, sin)
        ctx.kwargs = kwargs
        return (q_out, k_out) if k is not None else q_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk=None):
        q, k, q_weight, k_weight, q_rstd, k_rstd, cos, sin = ctx.saved_tensors
        need = ctx.needs_input_grad
        got = _op(_NORM_FWD, True)(dq, dk, q, k, q_weight, k_weight, q_rstd, k_rstd, cos, sin, **ctx.kwargs,
                                   weight_grads=[need[2], need[3]])
        return (got[0] if need[0] else None, got[1] if need[1] else None,
                got[2].to(q_weight.dtype) if need[2] else None, got[3].to(k_weight.dtype) if need[3] else None,
                None, None, None, None)


def norm_rotary(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                k_weight: Optional[torch.Tensor], cos: Optional[torch.Tensor], sin: Optional[torch.Tensor], *,
                rotary_mode: str = "interleave", partial_slice: Optional[Sequence[int]] = None,
                norm_slice: Optional[Sequence[int]] = None, eps: float = 1e-6):
    """Root-mean-square norm of the rows of ``q`` and ``k`` (which may be None) over
    the lanes ``norm_slice`` (default: all), times the weights, then the rotation
    of the lanes ``partial_slice`` (default: none); see
    ``binding.rope_partial_norm_fwd``.  Returns new tensors (q_out, k_out)."""
    register()
    ps = [0, 0] if partial_slice is None else [int(v) for v in partial_slice]
    ns = [0, q.shape[-1]] if norm_slice is None else [int(v) for v in norm_slice]
    _check_norm(q, k, rotary_mode, ps, ns)
    kwargs = dict(rotary_mode=rotary_mode, partial_slice=ps, norm_slice=ns)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, q_weight, k_weight)):
        got = NormRotaryFn.apply(q, k, q_weight, k_weight, cos, sin, kwargs, float(eps))
        return got if k is not None else (got, None)
    got = _op(_NORM_FWD, False)(q, k, q_weight, k_weight, cos, sin, **kwargs, eps=float(eps), keep_rstd=False)
    return got[0], got[1] if k is not None else None
