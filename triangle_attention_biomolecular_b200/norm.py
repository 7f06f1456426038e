"""Layer norm of pair rows and the 8-bit activation checkpoint.

``layer_norm(x, weight, bias)`` normalises the last dimension of a BF16 or FP32
tensor and is differentiable in all three.  With ``checkpoint="int8"`` or
``"e4m3"`` the forward keeps x in 8 bits (1.03 bytes a value in place of 2 or 4)
and the backward reads that form.  ``norm_linear`` puts the projection that
follows into the same autograd step, so that neither x nor the norm's output is
kept: the backward restores the output from the 8-bit x and the row statistics.
It saves memory; the norm and the product (torch.matmul) are launches of their own.

The 8-bit form (:class:`Act8`): 32 neighbouring channels share a power-of-two
scale, the least under which the block's largest magnitude fits the code range
(127 for int8, 448 for e4m3).  Restoring to BF16 adds no rounding.  A block
that holds an infinity or a NaN is restored as NaNs.

These functions run on the current stream of their tensors' device.  To capture
a training step into a CUDA graph, run the whole step (forward and backward)
once on a side stream first, and capture it with no autograd graph of an
earlier eager step on the same leaves still alive: autograd ties the
accumulation of a leaf's gradient to the stream of the oldest live graph, as
for any other operator.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B

_KINDS = {"int8": (B.TRI_ACT8_INT8, torch.int8), "e4m3": (B.TRI_ACT8_E4M3, torch.float8_e4m3fn)}


class Act8(NamedTuple):
    """An activation in 8 bits: codes of x's shape, exponent bytes [..., ceil(C/32)] and the
    dtype x had."""
    codes: torch.Tensor
    exps: torch.Tensor
    dtype: torch.dtype

    @property
    def kind(self) -> int:
        return B.TRI_ACT8_INT8 if self.codes.dtype == torch.int8 else B.TRI_ACT8_E4M3

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()


def _kind(name: str):
    try:
        return _KINDS[name]
    except (KeyError, TypeError):
        raise ValueError(f"checkpoint kind must be 'int8' or 'e4m3', got {name!r}") from None


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x itself if its rows can be walked as they lie (contiguous, or 2-D with unit channel
    stride), else as an [R, C] view or, where no view does, a contiguous copy."""
    if x.is_contiguous() or (x.dim() == 2 and x.stride(1) == 1):
        return x
    if x.dim() > 2 and x.stride(-1) == 1:
        try:
            return x.view(-1, x.shape[-1])
        except RuntimeError:
            pass
    return x.contiguous()


def _param(p: Optional[torch.Tensor]):
    return None if p is None else p.contiguous()


def _empty(x: torch.Tensor, dtype: Optional[torch.dtype]) -> torch.Tensor:
    """An uninitialised contiguous tensor of x's shape."""
    if x.is_contiguous() and (dtype is None or dtype is x.dtype):
        return torch.empty_like(x)
    return x.new_empty(x.shape, dtype=dtype)


def _empty8(x: torch.Tensor, kind: str):
    _, dt = _kind(kind)
    *lead, C = x.shape
    return Act8(x.new_empty(x.shape, dtype=dt), x.new_empty((*lead, (C + 31) // 32), dtype=torch.uint8), x.dtype)


def act8_pack(x: torch.Tensor, kind: str = "int8") -> Act8:
    """x (BF16 or FP32, [..., C]) in 8 bits."""
    x2 = _rows(x)
    B._rows(x2, "x")
    a = _empty8(x, kind)
    B.tri_act8_pack(x2, a.codes, a.exps, a.kind)
    return a


def act8_unpack(a: Act8, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The values a stands for, in ``dtype`` (default: the dtype that was packed)."""
    x = a.codes.new_empty(a.codes.shape, dtype=dtype or a.dtype)
    B.tri_act8_unpack(_rows(a.codes), _rows(a.exps), a.kind, x)
    return x


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None,
                 checkpoint: Optional[str] = None):
    """Returns (y, stats, kept): y of x's shape in ``out_dtype`` (default: x's dtype), stats FP32
    [2, rows] (means, reciprocal standard deviations), and kept, x as an :class:`Act8` written
    in the same pass (None without ``checkpoint``)."""
    x2 = _rows(x)
    geometry = B._rows(x2, "x")
    y = _empty(x, out_dtype)
    stats = x.new_empty((2, geometry[2]), dtype=torch.float32)
    a = None if checkpoint is None else _empty8(x, checkpoint)
    # y, stats and the 8-bit form are known to fit: only the caller's tensors are checked
    B._norm_fwd(x2, geometry, _param(weight), _param(bias), y, y.data_ptr(), geometry[3], stats.data_ptr(),
                B._NO_ACT8 if a is None else (a.codes.data_ptr(), geometry[3], a.exps.data_ptr(), a.exps.shape[-1], a.kind),
                eps, None)
    return y, stats, a


def norm_restore(kept: Act8, stats, weight=None, bias=None, out_dtype: Optional[torch.dtype] = None):
    """The norm's output from the 8-bit x and the statistics of :func:`norm_forward`."""
    y = kept.codes.new_empty(kept.codes.shape, dtype=out_dtype or kept.dtype)
    B.tri_norm_restore(_rows(kept.codes), _rows(kept.exps), kept.kind, stats, _param(weight), _param(bias), y)
    return y


def norm_backward(x, stats, dy, weight=None, need_dx: bool = True, need_dw: Optional[bool] = None):
    """Returns (dx, dweight, dbias) for the upstream gradient dy; ``x`` is the forward's input or
    the :class:`Act8` it kept.  dx has x's dtype; dweight and dbias are FP32 [C] (None unless
    ``need_dw``, by default when there is a weight)."""
    dy2 = _rows(dy)
    geometry = B._rows(dy2, "dy")
    _, _, R, C = geometry
    dx = dw = db = None
    into = [0, 0, 0, 0, 0, 0]  # dx and its row stride, dw, db, workspace and its size
    if need_dx:
        dx = _empty(dy, x.dtype)
        into[0], into[1] = dx.data_ptr(), C
    if weight is not None if need_dw is None else need_dw:
        dw, db = dy.new_empty(C, dtype=torch.float32), dy.new_empty(C, dtype=torch.float32)
        need = B.tri_norm_bwd_workspace_bytes(R, C)
        ws = dy.new_empty(need, dtype=torch.uint8)
        into[2:] = dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need
    if isinstance(x, Act8):
        B._norm_bwd(None, _rows(x.codes), _rows(x.exps), x.kind, stats, _param(weight), dy2, geometry, x.dtype, into, None)
    else:
        B._norm_bwd(_rows(x), None, None, 0, stats, _param(weight), dy2, geometry, x.dtype, into, None)
    return dx, dw, db


def _save(ctx, x, kept, stats, *more):
    """Keeps x, or its 8-bit form in place of it."""
    ctx.x_dtype = None if kept is None else kept.dtype
    first = (x,) if kept is None else (kept.codes, kept.exps)
    ctx.save_for_backward(*first, stats, *more)


def _saved(ctx):
    s = ctx.saved_tensors
    if ctx.x_dtype is None:
        return s
    return (Act8(s[0], s[1], ctx.x_dtype), *s[2:])


def _like(g, p):
    return None if p is None else g.to(p.dtype)


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype, checkpoint):
        y, stats, kept = norm_forward(x, weight, bias, eps, out_dtype, checkpoint)
        _save(ctx, x, kept, stats, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, stats, weight, bias = _saved(ctx)
        need = ctx.needs_input_grad
        dx, dw, db = norm_backward(x, stats, dy, weight, need[0], need[1] or need[2])
        return dx, _like(dw, weight) if need[1] else None, _like(db, bias) if need[2] else None, None, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None,
               checkpoint: Optional[str] = None):
    """Differentiable layer norm over the last dimension (BF16 or FP32 in, ``out_dtype`` out).
    ``checkpoint`` "int8" or "e4m3" keeps x in 8 bits for the backward."""
    if checkpoint is not None:
        _kind(checkpoint)
    return LayerNormFunction.apply(x, weight, bias, eps, out_dtype, checkpoint)


def _product(a, b):
    """a @ b in their own dtype, whatever an autocast around the call says."""
    with torch.autocast(a.device.type, enabled=False):
        return torch.matmul(a, b)


class NormLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, proj, eps, checkpoint):
        y, stats, kept = norm_forward(x, weight, bias, eps, proj.dtype, checkpoint)
        _save(ctx, x, kept, stats, weight, bias, proj)
        ctx.eps = eps
        return _product(y, proj.t())

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, stats, weight, bias, proj = _saved(ctx)
        g = g.to(proj.dtype)
        need = ctx.needs_input_grad
        dx = dw = db = dproj = None
        if need[3]:
            if isinstance(x, Act8):
                y = norm_restore(x, stats, weight, bias, proj.dtype)
            else:
                y = norm_forward(x, weight, bias, ctx.eps, proj.dtype)[0]
            dproj = _product(g.reshape(-1, g.shape[-1]).t(), y.view(-1, y.shape[-1]))
        if need[0] or need[1] or need[2]:
            dx, dw, db = norm_backward(x, stats, _product(g, proj), weight, need[0], need[1] or need[2])
        return (dx, _like(dw, weight) if need[1] else None, _like(db, bias) if need[2] else None, dproj, None, None)


def norm_linear(x, weight, bias, proj, eps: float = 1e-5, checkpoint: Optional[str] = "int8"):
    """layer_norm(x) @ proj.T, differentiable in x, weight, bias and proj ([out, C], BF16 or FP32;
    it sets the dtype of the norm's output and of the result).  Between the passes only x is
    kept, in 8 bits unless ``checkpoint`` is None; the norm's output is computed again."""
    if checkpoint is not None:
        _kind(checkpoint)
    return NormLinearFunction.apply(x, weight, bias, proj, eps, checkpoint)
