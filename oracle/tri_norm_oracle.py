"""FP64 layer norm, 8-bit activation form and relative position bias, in numpy, from
their definitions; shares nothing with the CUDA path.

Layer norm of x [R, C]:  mean, rstd = 1/sqrt(var + eps), y = (x - mean) rstd w + b, and its
gradients.  8-bit form: blocks of 32 channels, scale 2^e with the least e >= -126 for which the
block's largest magnitude is at most Q 2^e (Q = 127 int8, 448 e4m3).  Relative position bias: the
bucket of a pair is the number of edges not above pos_k - pos_q, or one past the last for pairs
of different groups.
"""
import numpy as np


def fwd(x, w, b, eps):
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    h = (x - mean) * rstd
    return h * (1.0 if w is None else w) + (0.0 if b is None else b), mean[:, 0], rstd[:, 0]


def bwd(x, mean, rstd, w, dy):
    """Gradients for given statistics (those of the forward's input, while x may be its 8-bit
    form): dx, dw, db."""
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


Q = {"int8": 127.0, "e4m3": 448.0}


def e4m3_round(v):
    """Nearest e4m3 value (ties to even) of |v| <= 448."""
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(v / step) * step


def act8(x, kind):
    """(codes as numbers, exponent bytes, restored values) of x [R, C] (float64)."""
    R, C = x.shape
    codes, vals = np.zeros((R, C)), np.zeros((R, C))
    exps = np.zeros((R, (C + 31) // 32), np.uint8)
    for j in range(exps.shape[1]):
        blk = x[:, 32 * j:32 * j + 32]
        sl = slice(32 * j, 32 * j + blk.shape[1])
        for r in range(R):
            amax = np.abs(blk[r]).max()
            if not np.isfinite(amax):
                exps[r, j], vals[r, sl] = 255, np.nan
                continue
            e = -126
            while amax > Q[kind] * 2.0 ** e:
                e += 1
            u = blk[r] * 2.0 ** -e
            codes[r, sl] = np.rint(u) if kind == "int8" else e4m3_round(u)
            exps[r, j], vals[r, sl] = e + 127, codes[r, sl] * 2.0 ** e
    return codes, exps, vals


def buckets(edges, pos_q, pos_k, group_q=None, group_k=None):
    """int64 [B, Nq, Nk]."""
    delta = pos_k.astype(np.int64)[:, None, :] - pos_q.astype(np.int64)[:, :, None]
    out = (delta[..., None] >= np.asarray(edges, np.int64)).sum(-1)
    if group_q is not None:
        out[group_q[:, :, None] != group_k[:, None, :]] = len(edges) + 1
    return out


def relpos_fwd(table, bucket, base=None):
    bias = np.moveaxis(table[bucket], -1, 1)
    return bias if base is None else bias + base


def relpos_bwd(dbias, bucket, nb):
    out = np.zeros((nb, dbias.shape[1]))
    for h in range(dbias.shape[1]):
        np.add.at(out[:, h], bucket.ravel(), dbias[:, h].ravel())
    return out
