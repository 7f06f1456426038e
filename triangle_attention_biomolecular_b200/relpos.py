"""Learned relative position bias for the attention's bias input.

A distance ``pos_k[b, j] - pos_q[b, i]`` falls into the bucket counted by the
edges that are not above it (``edges`` ascending, int32, above -2**31), and the
bias is that row of a learned table; with groups (chains, segments) a pair of
different groups takes the table's last row.  :func:`relpos_edges_clipped` and
:func:`relpos_edges_log` build the two usual sets of edges.

``relative_position_bias`` returns BF16 [B, H, Nq, Nk] in the padded layout that
``triangle_attention`` reads, is differentiable in the table and in ``base`` (a
bias to add to, such as a projected pair bias), and gives the table's gradient
in one pass over the bias's, with no atomics: repeated runs are bitwise equal.
To capture a training step into a CUDA graph, run it once on a side stream first,
and with no autograd graph of an earlier eager step on the same leaves alive, as
for the norm.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B


def relpos_edges_clipped(r: int, device="cuda") -> torch.Tensor:
    """Edges of 2 r + 1 buckets: each distance from -r to r its own, farther ones with the ends."""
    if not 1 <= r <= 255:
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE, f"r must be from 1 to 255, got {r}")
    return torch.arange(1 - r, r + 1, dtype=torch.int32, device=device)


def relpos_edges_log(per_side: int, max_distance: int, device="cuda") -> torch.Tensor:
    """Edges of 2 * per_side + 1 buckets: distance 0, and per_side buckets to either side, the
    first half of them one distance each, the others growing geometrically up to the last,
    which starts at max_distance.  With per_side 1 the one bucket of a side is the last one, and
    the nearer distances fall into that of distance 0."""
    if not 1 <= per_side <= 255 or not per_side <= max_distance < 2 ** 31:
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE,
                             f"1 <= per_side <= 255 and per_side <= max_distance < 2**31 are needed, got {per_side}, {max_distance}")
    exact = (per_side + 1) // 2
    steps = per_side - exact
    up = list(range(1, exact + 1)) if steps else [max_distance]
    for k in range(1, steps + 1):
        # least n with (n / exact)^steps >= (max_distance / exact)^k, in whole numbers
        n = int(exact * (max_distance / exact) ** (k / steps))
        bound = exact ** (steps - k) * max_distance ** k
        while n ** steps >= bound:
            n -= 1
        while n ** steps < bound:
            n += 1
        up.append(max(n, up[-1] + 1))
    return torch.tensor([1 - u for u in reversed(up)] + up, dtype=torch.int32, device=device)


def _layout(t: torch.Tensor) -> torch.Tensor:
    """t itself if the C ABI accepts its layout (unit inner stride, the others non-negative
    multiples of 8, 16-byte aligned data that reach to the end of the last row's last 16 bytes),
    else a copy with rows padded to a multiple of 8."""
    if t.dtype is not torch.bfloat16:
        raise B.TriAttnError(B.TRI_ATTN_ERR_DTYPE, f"a bias or its gradient must be torch.bfloat16, got {t.dtype}")
    b, h, q, n = t.shape
    sb, sh, sq, sn = t.stride()
    sb, sh, sq = sb if b > 1 else 0, sh if h > 1 else 0, sq if q > 1 else 0
    if not (t.data_ptr() % 16 or sb % 8 or sh % 8 or sq % 8) and (sn == 1 or n == 1):
        end = (b - 1) * sb + (h - 1) * sh + (q - 1) * sq + (n + 7) // 8 * 8
        if n % 8 == 0 or 2 * (t.storage_offset() + end) <= t.untyped_storage().nbytes():
            return t
    return _padded(t.shape, t).copy_(t)


def _padded(shape, like) -> torch.Tensor:
    """An uninitialised BF16 tensor whose rows are padded to a multiple of 8.  It is cut to its
    shape in place: were it a view, autograd would refuse in-place changes of a bias that a
    Function returns."""
    *lead, n = shape
    if n % 8 == 0:
        return like.new_empty(shape, dtype=torch.bfloat16)
    t = like.new_empty((*lead, (n + 7) // 8 * 8), dtype=torch.bfloat16)
    return t.as_strided_(shape, t.stride())


def _index(pos_q, pos_k, group_q, group_k, like=None):
    """Positions and groups as int32 [B, N], one batch size (that of ``like`` where all are shared),
    groups laid out as the positions."""
    if pos_q.dim() == 2 and pos_q.is_contiguous() and pos_k.dim() == 2 and pos_k.is_contiguous():
        n = pos_q.shape[0]
        if n == pos_k.shape[0] and (like is None or like.shape[0] == n) and (
                group_q is None or group_k is None
                or (group_q.shape == pos_q.shape and group_q.is_contiguous()
                    and group_k.shape == pos_k.shape and group_k.is_contiguous())):
            return pos_q, pos_k, group_q, group_k  # checked further where they are used
    ts = [pos_q, pos_k, group_q, group_k]
    for t in ts:
        if t is not None and (t.dtype != torch.int32 or not 1 <= t.dim() <= 2):
            raise B.TriAttnError(B.TRI_ATTN_ERR_DTYPE, f"positions and groups are int32 [N] or [B, N], got {t.dtype} {list(t.shape)}")
    ts = [t if t is None or t.dim() == 2 else t[None] for t in ts]
    n = max([t.shape[0] for t in ts if t is not None] + ([] if like is None else [like.shape[0]]))
    if any(t is not None and t.shape[0] not in (1, n) for t in ts):
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE, "positions and groups of different batch sizes")
    out = []
    for p, g in ((ts[0], ts[2]), (ts[1], ts[3])):
        p = p.expand(n, -1)
        if g is not None:
            g = g.expand(n, -1)
            if g.stride() != p.stride():
                p, g = p.contiguous(), g.contiguous()
        if p.stride(1) != 1:
            p, g = p.contiguous(), None if g is None else g.contiguous()
        out.append((p, g))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def relpos_forward(table, edges, pos_q, pos_k, group_q=None, group_k=None, base=None):
    """The bias, BF16 [B, H, Nq, Nk] with rows padded to a multiple of 8 elements.  table BF16 or
    FP32 [buckets, H]; positions and groups int32 [N] or [B, N]; base BF16 [B, H, Nq, Nk]."""
    if table.dim() != 2:
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE, f"table must be [buckets, H], got {list(table.shape)}")
    if base is not None and base.dim() != 4:
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE, f"base must be [B, H, Nq, Nk], got {list(base.shape)}")
    q, k, gq, gk = _index(pos_q, pos_k, group_q, group_k, base)
    bias = _padded((q.shape[0], table.shape[1], q.shape[1], k.shape[1]), table)
    B.tri_relpos_fwd(table.contiguous(), edges, q, k, gq, gk, None if base is None else _layout(base), bias)
    return bias


def relpos_backward(dbias, edges, pos_q, pos_k, group_q=None, group_k=None):
    """The table's gradient, FP32 [buckets, H], for the bias's gradient (BF16 [B, H, Nq, Nk])."""
    if dbias.dim() != 4:
        raise B.TriAttnError(B.TRI_ATTN_ERR_SHAPE, f"dbias must be [B, H, Nq, Nk], got {list(dbias.shape)}")
    q, k, gq, gk = _index(pos_q, pos_k, group_q, group_k, dbias)
    E, H = edges.numel(), dbias.shape[1]  # their shape is checked with the others
    dtable = dbias.new_empty((E + 1 + (gq is not None), H), dtype=torch.float32)
    ws = dbias.new_empty(B.tri_relpos_bwd_workspace_bytes(q.shape[0], H, q.shape[1], k.shape[1], E, gq is not None),
                         dtype=torch.uint8)
    B.tri_relpos_bwd(_layout(dbias), edges, q, k, gq, gk, dtable, ws)
    return dtable


class RelativePositionBiasFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, base, edges, pos_q, pos_k, group_q, group_k):
        ctx.save_for_backward(edges, pos_q, pos_k, group_q, group_k)
        ctx.table_dtype = table.dtype
        return relpos_forward(table, edges, pos_q, pos_k, group_q, group_k, base)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        dtable = None
        if ctx.needs_input_grad[0]:
            dtable = relpos_backward(g, *ctx.saved_tensors).to(ctx.table_dtype)
        return dtable, g if ctx.needs_input_grad[1] else None, None, None, None, None, None


def relative_position_bias(table, edges, pos_q, pos_k=None, group_q=None, group_k=None,
                           base: Optional[torch.Tensor] = None):
    """Differentiable relative position bias (see :func:`relpos_forward`).  Without ``pos_k`` the
    keys have the queries' positions, and their groups unless ``group_k`` gives others."""
    if pos_k is None:
        pos_k, group_k = pos_q, group_q if group_k is None else group_k
    return RelativePositionBiasFunction.apply(table, base, edges, pos_q, pos_k, group_q, group_k)
