"""Layer norm (tri_norm_fwd, tri_norm_restore, tri_norm_bwd) and the 8-bit activation form
(tri_act8_pack, tri_act8_unpack): host-side checks (no GPU) and GPU parity against the FP64
oracle (oracle/tri_norm_oracle.py) on the same inputs."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import triangle_attention_biomolecular_b200 as T
from oracle import tri_norm_oracle as O
from triangle_attention_biomolecular_b200 import _binding as Bd
from triangle_attention_biomolecular_b200 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                              # half a step of FP32, relative
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}     # half a step of the output's type


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return Bd.load()


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------
def test_struct_layout_matches_the_header():
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "tri_attn.h"
int main(void){
  printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu\n", sizeof(tri_act8_args), offsetof(tri_act8_args, x_type),
         sizeof(tri_act8), sizeof(tri_norm_fwd_args),
         offsetof(tri_norm_fwd_args, act), offsetof(tri_norm_fwd_args, C), offsetof(tri_norm_fwd_args, eps),
         sizeof(tri_norm_bwd_args), offsetof(tri_norm_bwd_args, workspace));
  return 0; }
'''
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    N, W = Bd.NormFwdArgs, Bd.NormBwdArgs
    assert got == [ctypes.sizeof(Bd.Act8Args), Bd.Act8Args.x_type.offset, ctypes.sizeof(Bd.Act8), ctypes.sizeof(N), N.act.offset, N.C.offset, N.eps.offset, ctypes.sizeof(W),
                   W.workspace.offset]


def fake(R=300, C=128, base=0x10000):
    """Aligned but fake pointers: every case is rejected before anything could use them."""
    a = Bd.NormFwdArgs()
    a.R, a.C, a.eps = R, C, 1e-5
    a.x, a.w, a.b, a.y, a.stats, a.act.codes, a.act.exps = (base + k * 0x1000000 for k in range(7))
    a.x_stride = a.y_stride = a.act.codes_stride = C
    a.act.exps_stride, a.act.kind = (C + 31) // 32, Bd.TRI_ACT8_INT8
    return a


def fake_bwd(**kw):
    a = Bd.NormBwdArgs()
    a.f = fake(**kw)
    a.dy, a.dx, a.dw, a.db, a.workspace = (0x8000000 + k * 0x1000000 for k in range(5))
    a.dy_stride = a.dx_stride = a.f.C
    a.workspace_bytes = Bd.tri_norm_bwd_workspace_bytes(a.f.R, a.f.C)
    return a


def status(fn, a, **change):
    for k, v in change.items():
        obj, names = a, k.split("__")
        for n in names[:-1]:
            obj = getattr(obj, n)
        setattr(obj, names[-1], v)
    return fn(bytes(a), None)


FWD_REFUSALS = [
    ({"x": None}, Bd.TRI_ATTN_ERR_NULL), ({"y": None}, Bd.TRI_ATTN_ERR_NULL), ({"stats": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"act__codes": None}, Bd.TRI_ATTN_ERR_NULL), ({"act__exps": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"R": -1}, Bd.TRI_ATTN_ERR_SHAPE), ({"C": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"C": 8193}, Bd.TRI_ATTN_ERR_UNSUPPORTED),
    ({"eps": -1.0}, Bd.TRI_ATTN_ERR_SHAPE), ({"eps": float("nan")}, Bd.TRI_ATTN_ERR_SHAPE),
    ({"x_type": 2}, Bd.TRI_ATTN_ERR_DTYPE), ({"y_type": -1}, Bd.TRI_ATTN_ERR_DTYPE), ({"w_type": 7}, Bd.TRI_ATTN_ERR_DTYPE),
    ({"act__kind": 3}, Bd.TRI_ATTN_ERR_UNSUPPORTED), ({"y_stride": 127}, Bd.TRI_ATTN_ERR_STRIDE),
    ({"x_stride": -128}, Bd.TRI_ATTN_ERR_STRIDE), ({"act__codes_stride": 127}, Bd.TRI_ATTN_ERR_STRIDE),
    ({"act__exps_stride": 3}, Bd.TRI_ATTN_ERR_STRIDE), ({"x": 0x10001}, Bd.TRI_ATTN_ERR_ALIGN),
    ({"y_type": 1, "y": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN), ({"stats": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN),
    ({"w_type": 1, "b": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN),
]


@pytest.mark.parametrize("change,want", FWD_REFUSALS)
def test_fwd_refusals(lib, change, want):
    assert status(lib.tri_norm_fwd, fake(), **change) == want


BWD_REFUSALS = [
    ({"dy": None}, Bd.TRI_ATTN_ERR_NULL), ({"dw": None}, Bd.TRI_ATTN_ERR_NULL), ({"f__stats": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"f__act__kind": 0, "f__x": None}, Bd.TRI_ATTN_ERR_NULL), ({"f__act__codes": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"f__C": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"f__R": -5}, Bd.TRI_ATTN_ERR_SHAPE), ({"f__x_type": 9}, Bd.TRI_ATTN_ERR_DTYPE),
    ({"dx_stride": 64}, Bd.TRI_ATTN_ERR_STRIDE), ({"dy_stride": -1}, Bd.TRI_ATTN_ERR_STRIDE),
    ({"db": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN), ({"workspace": None}, Bd.TRI_ATTN_ERR_WORKSPACE),
    ({"workspace_bytes": 64}, Bd.TRI_ATTN_ERR_WORKSPACE), ({"workspace": 0x10004}, Bd.TRI_ATTN_ERR_ALIGN),
]


@pytest.mark.parametrize("change,want", BWD_REFUSALS)
def test_bwd_refusals(lib, change, want):
    assert status(lib.tri_norm_bwd, fake_bwd(), **change) == want


def test_restore_and_act8_refusals(lib):
    assert lib.tri_norm_fwd(None, None) == lib.tri_norm_bwd(None, None) == lib.tri_norm_restore(None, None) == Bd.TRI_ATTN_ERR_NULL
    assert status(lib.tri_norm_restore, fake(), act__kind=0) == Bd.TRI_ATTN_ERR_UNSUPPORTED
    assert status(lib.tri_norm_restore, fake(), act__codes=None) == Bd.TRI_ATTN_ERR_NULL
    assert lib.tri_act8_pack(None, None) == lib.tri_act8_unpack(None, None) == Bd.TRI_ATTN_ERR_NULL
    for fn, what, want in (
            (lib.tri_act8_pack, {"R": -1}, Bd.TRI_ATTN_ERR_SHAPE), (lib.tri_act8_pack, {"C": 0}, Bd.TRI_ATTN_ERR_SHAPE),
            (lib.tri_act8_unpack, {"C": 2 ** 30 + 1}, Bd.TRI_ATTN_ERR_SHAPE),
            (lib.tri_act8_pack, {"x": None}, Bd.TRI_ATTN_ERR_NULL), (lib.tri_act8_pack, {"x_type": 5}, Bd.TRI_ATTN_ERR_DTYPE),
            (lib.tri_act8_pack, {"act__codes_stride": 127}, Bd.TRI_ATTN_ERR_STRIDE),  # code rows would overlap
            (lib.tri_act8_pack, {"act__exps": None}, Bd.TRI_ATTN_ERR_NULL),
            (lib.tri_act8_unpack, {"x_stride": 100}, Bd.TRI_ATTN_ERR_STRIDE),
            (lib.tri_act8_unpack, {"x": 0x10001}, Bd.TRI_ATTN_ERR_ALIGN),
            (lib.tri_act8_unpack, {"act__kind": 0}, Bd.TRI_ATTN_ERR_UNSUPPORTED)):
        a = Bd.Act8Args()
        a.R, a.C, a.x, a.x_stride, a.act = 8, 128, 0x3000000, 128, Bd.Act8(0x10000, 128, 0x2000000, 4, 1)
        assert status(fn, a, **what) == want


def test_workspace_bytes(lib):
    assert Bd.tri_norm_bwd_workspace_bytes(10, 0) == 0 and Bd.tri_norm_bwd_workspace_bytes(-1, 8) == 0
    assert Bd.tri_norm_bwd_workspace_bytes(10, 8193) == 0
    for C in (1, 128, 512, 513, 8192):
        small, big, huge = (Bd.tri_norm_bwd_workspace_bytes(R, C) for R in (1, 10 ** 6, 10 ** 12))
        assert 0 < small <= big == huge and big % (2 * 4 * C) == 0
        assert Bd.tri_norm_bwd_workspace_bytes(0, C) > 0


def test_python_refusals_on_cpu(lib):
    x = torch.zeros(4, 128, dtype=BF)
    for scalar in (lambda t: T.norm_forward(t), lambda t: T.act8_pack(t), lambda t: T.layer_norm(t)):
        with pytest.raises(Bd.TriAttnError) as e:
            scalar(torch.tensor(1.0))
        assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE
    for call in (lambda: T.norm_forward(x), lambda: T.act8_pack(x), lambda: T.layer_norm(x)):
        with pytest.raises(Bd.TriAttnError, match="CUDA device"):
            call()
    with pytest.raises(Bd.TriAttnError) as e:
        T.norm_forward(x.half())
    assert e.value.status == Bd.TRI_ATTN_ERR_DTYPE
    with pytest.raises(Bd.TriAttnError) as e:
        T.norm_forward(x, torch.zeros(127))
    assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE
    with pytest.raises(Bd.TriAttnError) as e:
        T.norm_forward(x, torch.zeros(128), torch.zeros(128, dtype=BF))
    assert e.value.status == Bd.TRI_ATTN_ERR_DTYPE
    with pytest.raises(Bd.TriAttnError) as e:
        T.norm_forward(torch.zeros(3, 0))
    assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE
    with pytest.raises(ValueError, match="int8"):
        T.layer_norm(x, checkpoint="int4")
    with pytest.raises(Bd.TriAttnError) as e:  # statistics of another number of rows
        T.norm_backward(x, torch.zeros(2, 3), x)
    assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE
    with pytest.raises(Bd.TriAttnError) as e:  # an upstream gradient of another shape
        T.norm_backward(x, torch.zeros(2, 5), torch.zeros(5, 128, dtype=BF))
    assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE


# ---------------------------------------------------------------------------
# GPU parity
# ---------------------------------------------------------------------------
# Bounds, per element, u = 2^-24.  A row's sums add at most 16 + 5 terms one after another (plus
# 16 across warps), so mean is off by < 40 u max|x|, and x - mean with it; the variance is a sum of
# squares (relative error < 45 u, the mean's error enters squared), rstd adds 2 steps.  Hence
#   |h - h_ref| < 128 u X,  X = rstd max|x|,   |y - y_ref| < half |y| + 128 u (X |w| + |b|).
# dx = rstd (g - c1 - h c2) with |c1| <= M = max|g|, |c2| <= M Hm, Hm = max|h|:
#   < half |dx| + 128 u rstd M (1 + Hm^2 + 2 Hm X).
# dw, db add per thread the rows it owns (< 64 at these sizes), then < 64 more partial sums:
#   < 128 u sum |dy h| + sum 128 u X |dy|   and   < 128 u sum |dy|.
def make(R, C, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * (0.5 + 2 * torch.rand(C, generator=g)) + torch.randn(C, generator=g)
    out = torch.full((R, C + pad), float("nan"), dtype=dtype, device="cuda")
    out[:, :C] = x.to(dtype)
    return out[:, :C]


def f64(t):
    return t.detach().double().cpu().numpy()


def check_norm(x, xk, w, b, stats, y, again, dy, dx, dw, db, eps=1e-5):
    """y, statistics, the restored y and the gradients against the oracle; xk: the values the
    backward worked on."""
    X, W, Bv = f64(x), None if w is None else f64(w), None if b is None else f64(b)
    ref, mean, rstd = O.fwd(X, W, Bv, eps)
    aw, ab = (1.0 if W is None else np.abs(W)), (0.0 if Bv is None else np.abs(Bv))
    big = np.abs(X).max(1, initial=0)
    Xr = (rstd * big)[:, None]
    assert np.all(np.abs(f64(stats[0]) - mean) <= 40 * U * big)
    assert np.all(np.abs(f64(stats[1]) - rstd) <= 64 * U * rstd * (1 + rstd * big * 40 * U))
    assert np.all(np.abs(f64(y) - ref) <= HALF[y.dtype] * np.abs(ref) + 128 * U * (Xr * aw + ab))
    K = f64(xk)
    h = (K - mean[:, None]) * rstd[:, None]
    if again is not None:
        ref = h * (1.0 if W is None else W) + (0.0 if Bv is None else Bv)
        Xk = (rstd * np.maximum(big, np.abs(K).max(1, initial=0)))[:, None]
        assert np.all(np.abs(f64(again) - ref) <= HALF[again.dtype] * np.abs(ref) + 128 * U * (Xk * aw + ab + np.abs(h) * aw))
        Xr = Xk
    D = f64(dy)
    rdx, rdw, rdb = O.bwd(K, mean, rstd, W, D)
    M = np.abs(D * aw).max(1, initial=0)[:, None]
    Hm = np.abs(h).max(1, initial=0)[:, None]
    if dx is not None:
        assert np.all(np.abs(f64(dx) - rdx) <= HALF[dx.dtype] * np.abs(rdx)
                      + 128 * U * rstd[:, None] * M * (1 + Hm ** 2 + 2 * Hm * Xr))
    if dw is not None:
        assert np.all(np.abs(f64(dw) - rdw) <= 128 * U * (np.abs(D * h) + (Xr + np.abs(h)) * np.abs(D)).sum(0))
        assert np.all(np.abs(f64(db) - rdb) <= 128 * U * np.abs(D).sum(0))


CASES = [  # R, C, x, y, weight (None: no affine), padding of the rows
    (1, 128, BF, BF, F32, 0), (5, 128, BF, BF, BF, 0), (4099, 128, BF, BF, F32, 0), (4097, 128, F32, BF, F32, 16),
    (300, 128, BF, F32, None, 16), (300, 128, F32, F32, F32, 1), (77, 1, BF, BF, F32, 0), (77, 2, F32, F32, F32, 0),
    (129, 16, BF, BF, F32, 0), (129, 17, F32, BF, BF, 0), (65, 31, BF, BF, F32, 0), (65, 32, F32, F32, F32, 0),
    (65, 33, BF, F32, F32, 0), (64, 48, BF, BF, None, 0), (64, 112, F32, F32, F32, 0), (50, 255, BF, BF, F32, 0),
    (70, 100, BF, BF, F32, 0), (1300, 67, F32, BF, BF, 0), (900, 200, F32, F32, F32, 0), (50, 387, F32, F32, F32, 0), (50, 384, BF, BF, F32, 0), (33, 512, BF, BF, F32, 0), (33, 513, BF, BF, F32, 0),
    (33, 528, F32, F32, BF, 0), (700, 1024, BF, BF, F32, 0), (20, 1025, F32, BF, F32, 0), (9, 8192, BF, BF, F32, 0),
    (9, 8191, F32, F32, F32, 3), (3000, 640, BF, BF, F32, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [None, "int8", "e4m3"])
@pytest.mark.parametrize("R,C,xt,yt,wt,pad", CASES)
def test_parity(R, C, xt, yt, wt, pad, kept):
    x = make(R, C, xt, 7 * R + C, pad)
    w = b = None
    if wt is not None:
        w, b = (1 + 0.3 * make(1, C, F32, C)[0]).to(wt), make(1, C, F32, C + 1)[0].to(wt)
    dy = make(R, C, yt, R + 3 * C, pad)
    y, stats, a = T.norm_forward(x, w, b, out_dtype=yt, checkpoint=kept)
    assert y.dtype == yt and y.shape == x.shape and torch.isfinite(y).all()
    again, xk = None, x
    if kept:
        again = T.norm_restore(a, stats, w, b, out_dtype=yt)
        _, exps, vals = O.act8(f64(x), kept)
        np.testing.assert_array_equal(a.exps.cpu().numpy(), exps)
        xk = T.act8_unpack(a, F32)
        np.testing.assert_array_equal(f64(xk), vals)
    dx, dw, db = T.norm_backward(a if kept else x, stats, dy, w)
    assert (dw is None) == (w is None) and dx.dtype == xt
    check_norm(x, xk, w, b, stats, y, again, dy, dx, dw, db)
    # bitwise repeatable
    d2 = T.norm_backward(a if kept else x, stats, dy, w)
    assert torch.equal(dx, d2[0]) and (w is None or (torch.equal(dw, d2[1]) and torch.equal(db, d2[2])))


@pytest.mark.gpu
def test_long_sums_and_only_some_gradients():
    R, C = 200_003, 64
    x, dy = make(R, C, BF, 1), make(R, C, BF, 2)
    w = torch.ones(C, device="cuda")
    _, stats, _ = T.norm_forward(x, w)
    dx, dw, db = T.norm_backward(x, stats, dy, w)
    K, D = f64(x), f64(dy)
    _, mean, rstd = O.fwd(K, None, None, 1e-5)
    h = (K - mean[:, None]) * rstd[:, None]
    # a thread adds R / (296 blocks x 64 rows) < 16 rows, then < 64 partial sums
    assert np.all(np.abs(f64(dw) - (D * h).sum(0)) <= 128 * U * (np.abs(D) * (1 + 2 * np.abs(h) + (rstd * np.abs(K).max(1))[:, None])).sum(0))
    assert np.all(np.abs(f64(db) - D.sum(0)) <= 128 * U * np.abs(D).sum(0))
    none, dw2, db2 = T.norm_backward(x, stats, dy, w, need_dx=False)
    assert none is None and torch.equal(dw, dw2) and torch.equal(db, db2)
    dx3, dw3, db3 = T.norm_backward(x, stats, dy, w, need_dw=False)
    assert dw3 is None and db3 is None and torch.equal(dx, dx3)


@pytest.mark.gpu
def test_large_rows_past_32_bits():
    """Element offsets past 2^31: the last rows equal the same rows alone, in every direction."""
    R, C = 2 ** 24 + 77, 128
    x = torch.empty(R, C, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    w, b = 1 + 0.3 * make(1, C, F32, 1)[0], make(1, C, F32, 2)[0]
    y, stats, a = T.norm_forward(x, w, b, checkpoint="int8")
    again = T.norm_restore(a, stats, w, b)
    dx, dw, db = T.norm_backward(a, stats, y, w)
    tail = slice(R - 500, R)
    y1, s1, a1 = T.norm_forward(x[tail], w, b, checkpoint="int8")
    assert torch.equal(y[tail], y1) and torch.equal(stats[:, tail], s1)
    assert torch.equal(a.codes[tail], a1.codes) and torch.equal(a.exps[tail], a1.exps)
    assert torch.equal(again[tail], T.norm_restore(a1, s1, w, b))
    assert torch.equal(dx[tail], T.norm_backward(a1, s1, y1, w)[0])
    assert torch.equal(T.act8_unpack(a)[tail], T.act8_unpack(a1))
    # db: a thread adds R / (296 x 32) < 1800 rows, then < 64 partial sums
    want = torch.stack([c.double().sum(0) for c in y.split(2 ** 21)]).sum(0)
    size = torch.stack([c.double().abs().sum(0) for c in y.split(2 ** 21)]).sum(0)
    assert ((db.double() - want).abs() <= 1900 * U * size).all() and torch.isfinite(dw).all()


@pytest.mark.gpu
def test_empty_single_and_strided_rows():
    x = torch.empty(0, 128, dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    y, stats, a = T.norm_forward(x, w, checkpoint="int8")
    assert y.shape == x.shape and stats.shape == (2, 0)
    assert T.norm_restore(a, stats, w).shape == x.shape and T.act8_unpack(a).shape == x.shape
    dx, dw, db = T.norm_backward(a, stats, x, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()  # sums over nothing
    # one row given to all (stride 0), read only
    row = make(1, 128, BF, 5)
    y, stats, _ = T.norm_forward(row.expand(37, 128), w)
    assert torch.equal(y, y[:1].expand(37, 128))
    dx, dw, _ = T.norm_backward(row.expand(37, 128), stats, row.expand(37, 128), w)
    assert torch.equal(dx, dx[:1].expand(37, 128))
    # pair tensors of four and five dimensions, and a frame that no view flattens
    z = make(6 * 7, 96, F32, 8).reshape(1, 6, 7, 96)
    full = T.norm_forward(z, None, None)[0]
    t = T.norm_forward(z.transpose(1, 2), None, None)[0]
    assert t.shape == (1, 7, 6, 96) and torch.equal(t.transpose(1, 2), full)
    assert torch.equal(T.norm_forward(z[..., ::2].contiguous())[0], T.norm_forward(z[..., ::2])[0])


@pytest.mark.gpu
def test_outputs_leave_what_lies_around_them():
    R, C = 37, 100
    x = make(R, C, BF, 3)
    for shift in (0, 3):  # aligned rows of 112, and rows that start at an odd element
        y = torch.full((R + 2, 112 + shift), float("nan"), dtype=BF, device="cuda")
        codes = torch.full((R + 2, 112 + shift), 99, dtype=torch.int8, device="cuda")
        exps = torch.full((R + 2, 9), 77, dtype=torch.uint8, device="cuda")
        stats = torch.full((2 * R + 4,), float("nan"), device="cuda")
        Bd.tri_norm_fwd(x, None, None, y[1:-1, shift:shift + C], stats[2:-2].view(2, R), codes[1:-1, shift:shift + C],
                        exps[1:-1, 1:5], Bd.TRI_ACT8_INT8)
        assert torch.isfinite(y[1:-1, shift:shift + C]).all() and torch.isfinite(stats[2:-2]).all()
        y[1:-1, shift:shift + C] = float("nan")
        codes[1:-1, shift:shift + C] = 99
        exps[1:-1, 1:5] = 77
        assert torch.isnan(y).all() and (codes == 99).all() and (exps == 77).all()
        assert torch.isnan(stats[:2]).all() and torch.isnan(stats[-2:]).all()


@pytest.mark.gpu
def test_rows_that_are_constant_or_not_finite():
    x = make(6, 128, F32, 9).clone()
    x[1] = 3.25           # variance 0: the norm is the bias
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 0
    b = make(1, 128, F32, 4)[0]
    y, stats, a = T.norm_forward(x, torch.ones(128, device="cuda"), b, checkpoint="int8")
    assert torch.equal(y[1], b) and torch.equal(y[4], b)
    assert torch.isnan(y[2]).any() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[[0, 1, 4, 5]]).all()  # the rows next to them are not touched
    back = T.act8_unpack(a)
    assert torch.isnan(back[2, :32]).all() and torch.isfinite(back[2, 32:]).all()
    assert torch.isnan(back[3, :32]).all() and torch.isfinite(back[[0, 1, 4, 5]]).all()
    assert not back[4].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("C", [1, 15, 16, 31, 32, 33, 48, 64, 100, 128, 209, 1000, 10000])
def test_act8_is_exact(kind, dtype, C):
    """Exponents, codes and restored values equal the definition: no tolerance."""
    R = 40 if C < 500 else 6
    x = make(R, C, F32, C).cpu()
    q = O.Q[kind]
    x *= torch.exp2(torch.randint(-140, 110, (R, 1), generator=torch.Generator().manual_seed(C)).float())
    x[0] = 0
    x[1, C // 2] = q
    x[2, C // 3] = float(np.nextafter(np.float32(q), np.float32(1e9)))
    x[3] = torch.arange(C).float() / 2            # ties
    x[4, 0] = torch.finfo(F32).max
    x[5, C - 1] = float("-inf")
    x = x.to(dtype).cuda()
    a = T.act8_pack(x, kind)
    codes, exps, vals = O.act8(f64(x), kind)
    np.testing.assert_array_equal(a.exps.cpu().numpy(), exps)
    np.testing.assert_array_equal(a.codes.float().cpu().numpy(), codes)
    # FP32 holds every value but those rounded up to 2^128 (from the largest finite ones): infinite there
    np.testing.assert_array_equal(f64(T.act8_unpack(a, F32)), f64(torch.tensor(vals).float()))
    back = T.act8_unpack(a)
    assert back.dtype == dtype
    # BF16 holds every value of either code; only below its least normal value can it round
    ref = torch.tensor(vals).to(dtype)
    assert torch.equal(torch.nan_to_num(back.cpu(), nan=-1), torch.nan_to_num(ref, nan=-1))


@pytest.mark.gpu
def test_act8_strided_rows():
    x = make(50, 64, BF, 2, pad=16)
    big = torch.full((50, 100), 7, dtype=torch.int8, device="cuda")
    exps = torch.full((50, 5), 9, dtype=torch.uint8, device="cuda")
    for start in (16, 3):
        Bd.tri_act8_pack(x, big[:, start:start + 64], exps[:, 1:3], Bd.TRI_ACT8_INT8)
        a = T.act8_pack(x, "int8")
        assert torch.equal(big[:, start:start + 64], a.codes) and torch.equal(exps[:, 1:3], a.exps)
        out = torch.full((50, 80), float("nan"), dtype=BF, device="cuda")
        Bd.tri_act8_unpack(big[:, start:start + 64], exps[:, 1:3], Bd.TRI_ACT8_INT8, out[:, 5:69])
        assert torch.equal(out[:, 5:69], T.act8_unpack(a)) and torch.isnan(out[:, :5]).all() and torch.isnan(out[:, 69:]).all()
        big[:, start:start + 64] = 7
        assert (big == 7).all() and (exps[:, [0, 3, 4]] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [None, "int8"])
def test_autograd_against_differences(kept):
    """Gradients of a scalar of the FP32 norm against central differences of the FP64 formula."""
    R, C = 4, 40
    g = torch.Generator().manual_seed(11)
    x, w, b, s = (torch.randn(*n, generator=g) for n in ((R, C), (C,), (C,), (R, C)))
    xg, wg, bg = (t.cuda().requires_grad_() for t in (x, w, b))
    y = T.layer_norm(xg, wg, bg, checkpoint=kept)
    (y * s.cuda()).sum().backward()
    X, W, Bv, S = (t.double().numpy() for t in (x, w, b, s))
    f = lambda X, W, Bv: (O.fwd(X, W, Bv, 1e-5)[0] * S).sum()  # noqa: E731
    # differences: 1e-8; FP32: < 1e-5; with the 8-bit x: 2^-7 of a block's largest value, ~3, over
    # the row's spread, ~1, in h, and twice that in dx: 0.1
    tol = 1e-5 if kept is None else 0.1
    for k, (a, grad) in enumerate(((X, xg.grad), (W, wg.grad), (Bv, bg.grad))):
        got = f64(grad)
        assert grad.dtype == F32
        for i in np.ndindex(a.shape):
            d = np.zeros(a.shape)
            d[i] = 1e-5
            lo, hi = [X, W, Bv], [X, W, Bv]
            lo[k], hi[k] = a - d, a + d
            assert abs((f(*hi) - f(*lo)) / 2e-5 - got[i]) < tol * (1 + R * (k > 0))


@pytest.mark.gpu
def test_autograd_options():
    x = make(30, 128, BF, 1).clone().requires_grad_()
    w = torch.ones(128, device="cuda", dtype=BF, requires_grad=True)
    y = T.layer_norm(x, w, None, out_dtype=F32)
    assert y.dtype == F32
    y.sum().backward()  # a gradient of stride 0
    assert x.grad.dtype == BF and w.grad.dtype == BF
    x.grad = None
    T.layer_norm(x).float().square().sum().backward()  # no parameters
    assert x.grad is not None
    b = torch.zeros(128, device="cuda", requires_grad=True)
    T.layer_norm(x.detach(), None, b).sum().backward()  # the bias alone
    assert torch.equal(b.grad, torch.full_like(b, 30))
    with pytest.raises(RuntimeError):  # no second derivatives
        gx, = torch.autograd.grad(T.layer_norm(x, w).float().square().sum(), x, create_graph=True)
        gx.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("kept", ["int8", "e4m3"])
def test_checkpoint_keeps_8_bits_and_the_same_output(kept):
    x = make(64 * 64, 128, BF, 21).reshape(1, 64, 64, 128)
    w, b = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")
    x = x.clone().requires_grad_()
    y = T.layer_norm(x, w, b, checkpoint=kept)
    assert torch.equal(y, T.layer_norm(x, w, b))
    saved = [t for t in y.grad_fn.saved_tensors if t is not None and t.numel() >= x.numel() // 32]
    assert sum(t.numel() * t.element_size() for t in saved if t.dtype != F32) <= x.numel() * 33 // 32


@pytest.mark.gpu
def test_streams_and_graphs():
    x, dy = make(3000, 128, BF, 1), make(3000, 128, BF, 2)
    w = torch.ones(128, device="cuda")

    def step():
        y, stats, a = T.norm_forward(x, w, checkpoint="int8")
        return (y, T.norm_restore(a, stats, w), *T.norm_backward(a, stats, dy, w))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs of the same step, replayed in turn and with new inputs
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    x.copy_(make(3000, 128, BF, 5))
    want = step()
    for g, out in graphs + graphs:
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # an explicit stream handle
    y = torch.empty_like(x)
    stats = torch.empty(2, 3000, device="cuda")
    torch.cuda.synchronize()
    Bd.tri_norm_fwd(x, w, None, y, stats, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    torch.cuda.synchronize()
    Bd.tri_norm_fwd(x, w, None, y, stats, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


@pytest.mark.gpu
def test_captured_training_step():
    x = make(500, 128, F32, 1).clone().requires_grad_()
    w, b = (torch.ones(128, device="cuda", requires_grad=True) for _ in range(2))

    def step():
        for t in (x, w, b):
            t.grad = None
        T.layer_norm(x, w, b, checkpoint="int8").square().sum().backward()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    want = [t.grad.clone() for t in (x, w, b)]
    for t in (x, w, b):
        t.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    assert all(torch.equal(t.grad, v) for t, v in zip((x, w, b), want))


@pytest.mark.gpu
def test_norm_linear():
    """The fused step against layer_norm and a product, both ways of keeping x."""
    g = torch.Generator().manual_seed(4)
    x0 = make(9 * 11, 128, BF, 6).reshape(9, 11, 128)
    w0, b0 = (1 + 0.2 * torch.randn(128, generator=g)).cuda(), torch.randn(128, generator=g).cuda()
    p0 = (torch.randn(200, 128, generator=g) / 128 ** 0.5).to(BF).cuda()
    up = torch.randn(9, 11, 200, generator=g).to(BF).cuda()

    def grads(f):
        ts = [t.clone().requires_grad_() for t in (x0, w0, b0, p0)]
        out = f(*ts)
        out.backward(up)
        return out.detach(), [t.grad for t in ts]

    want, gw = grads(lambda x, w, b, p: torch.matmul(T.layer_norm(x, w, b), p.t()))
    out, gn = grads(lambda x, w, b, p: T.norm_linear(x, w, b, p, checkpoint=None))
    assert torch.equal(out, want)
    for a, c in zip(gn, gw):
        # the same products of the same numbers, in another order at most
        assert a.dtype == c.dtype and (a.float() - c.float()).norm() <= 2.0 ** -8 * c.float().norm()
    out, g8 = grads(lambda x, w, b, p: T.norm_linear(x, w, b, p))
    assert torch.equal(out, want)
    for a, c in zip(g8, gw):
        # codes are within 1/127 of a block's largest value, which is within 4 of its spread: rms
        # 4/127/sqrt(3) = 0.018 in h; dx holds h twice
        assert (a.float() - c.float()).norm() <= 0.04 * c.float().norm()
    # every combination of what needs a gradient
    for need in range(1, 16):
        ts = [t.clone().requires_grad_(bool(need >> k & 1)) for k, t in enumerate((x0, w0, b0, p0))]
        T.norm_linear(*ts).backward(up)
        for t, c in zip(ts, g8):
            assert (t.grad is None) if not t.requires_grad else torch.equal(t.grad, c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_linear_under_autocast(dtype):
    """The projection's dtype sets the result's, in both passes, whatever autocast says."""
    x = make(40, 128, BF, 6).clone().requires_grad_()
    p = (make(32, 128, F32, 7) / 11).to(dtype).requires_grad_()
    T.norm_linear(x, None, None, p).float().square().sum().backward()
    want, x.grad, dp, p.grad = x.grad, None, p.grad, None
    with torch.autocast("cuda", dtype=BF):
        out = T.norm_linear(x, None, None, p)
        assert out.dtype == dtype
        out.float().square().sum().backward()
    assert torch.equal(x.grad, want) and torch.equal(p.grad, dp)


@pytest.mark.gpu
def test_pending_device_error_stops_the_norm_too():
    x = make(10, 128, BF, 1)
    y = torch.full_like(x, float("nan"))
    stats = torch.empty(2, 10, device="cuda")
    Bd.tri_attn_set_wait_limit_ns(1_000_000)
    try:
        Bd.tri_attn_selftest_expire_wait()
        Bd.tri_norm_fwd(x, None, None, y, stats)
        torch.cuda.synchronize()
        assert torch.isnan(y).all()
        assert Bd.tri_attn_device_error(True)[0] == Bd.TRI_ATTN_ERR_DEVICE_TIMEOUT
    finally:
        Bd.tri_attn_set_wait_limit_ns(2_000_000_000)
        Bd.tri_attn_device_error(True)
    Bd.tri_norm_fwd(x, None, None, y, stats)
    assert torch.isfinite(y).all()


def test_weight_gradients_are_tensors_of_their_own(lib, monkeypatch):
    """Not two views of one: those share a version counter and refuse in-place changes."""
    def backward(x, codes, exps, kind, stats, w, dy, geometry, x_dtype, into, stream, *others):
        C = geometry[3]
        for k, at in enumerate(into[2:4]):
            ctypes.memmove(at, (ctypes.c_float * C)(*[k + 1.0] * C), 4 * C)

    monkeypatch.setattr(Bd, "_norm_bwd", backward)
    monkeypatch.setattr(Bd, "_norm_fwd", lambda *a: None)
    x, w, b = torch.randn(4, 8), torch.ones(8, requires_grad=True), torch.ones(8, requires_grad=True)
    _, dw, db = T.norm_backward(x, torch.zeros(2, 4), x, w)
    assert (dw == 1).all() and (db == 2).all() and dw.dtype == db.dtype == F32 and dw.shape == db.shape == (8,)
    assert dw.untyped_storage().data_ptr() != db.untyped_storage().data_ptr()
    dw.add_(0.5 * w)  # weight decay, say
    assert dw.requires_grad and not db.requires_grad
    T.layer_norm(x, w, b).sum().backward()
    product = (w.grad * torch.ones(8, requires_grad=True)).sum()
    b.grad.zero_()  # has nothing to do with w.grad, which the product keeps
    assert w.grad._version == 0
    product.backward()


# rows that are walked element by element, in each way that lanes share them (4 lanes, a warp with
# four, eight or sixteen channels per lane, a block), and rows in vectors: three rounds of rows per
# block and a last one that is not full, forward and backward.  A block's rows per round times the
# blocks of the largest grid: 28416, 5920, 4736, 3552 and 1184 rows forward, less backward.
ROUNDS = [  # R, C, x, y, padding of the rows
    (57011, 33, BF, BF, 0), (57011, 64, F32, BF, 1), (12011, 67, BF, F32, 0), (12011, 128, BF, BF, 1),
    (9511, 129, F32, F32, 0), (9511, 256, BF, BF, 3), (7211, 257, F32, BF, 0), (7211, 387, BF, BF, 0),
    (7211, 512, F32, F32, 1), (2411, 513, F32, F32, 0), (2411, 1025, BF, BF, 0), (2411, 1024, BF, F32, 1),
    (2411, 1024, BF, BF, 0), (38011, 128, F32, F32, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [None, "int8", "e4m3"])
@pytest.mark.parametrize("R,C,xt,yt,pad", ROUNDS)
def test_many_rounds_of_rows(R, C, xt, yt, pad, kept):
    x, dy = make(R, C, xt, 7 * R + C, pad), make(R, C, yt, R + 3 * C, pad)
    w, b = 1 + 0.3 * make(1, C, F32, C)[0], make(1, C, F32, C + 1)[0]
    y, stats, a = T.norm_forward(x, w, b, out_dtype=yt, checkpoint=kept)
    again, xk = None, x
    if kept:
        again, xk = T.norm_restore(a, stats, w, b, out_dtype=yt), T.act8_unpack(a, F32)
        packed = T.act8_pack(x, kept)
        assert torch.equal(packed.codes.view(torch.uint8), a.codes.view(torch.uint8)) and torch.equal(packed.exps, a.exps)
    dx, dw, db = T.norm_backward(a if kept else x, stats, dy, w)
    # a thread adds 4 rows at most here, then the partial sums: within check_norm's counts
    check_norm(x, xk, w, b, stats, y, again, dy, dx, dw, db)
    # the same rows in calls of one round, bit for bit
    step = {True: 592, False: 2368}[C > 512]
    for r in range(0, R, step):
        s = slice(r, min(R, r + step))
        y1, s1, a1 = T.norm_forward(x[s], w, b, out_dtype=yt, checkpoint=kept)
        assert torch.equal(y[s], y1) and torch.equal(stats[:, s], s1)
        if kept:
            assert torch.equal(a.codes[s].view(torch.uint8), a1.codes.view(torch.uint8)) and torch.equal(a.exps[s], a1.exps)
            assert torch.equal(again[s], T.norm_restore(a1, s1, w, b, out_dtype=yt))
            assert torch.equal(xk[s], T.act8_unpack(a1, F32))
        assert torch.equal(dx[s], T.norm_backward(a1 if kept else x[s], s1, dy[s], w, need_dw=False)[0])


def guarded(R, C, dtype, fill, align):
    """A buffer full of ``fill`` and the [R, C] rows within it that a call may write: rows of a
    multiple of 32 bytes with something before and behind each, or rows at an odd element."""
    width = (C + 31) // 32 * 32 + 64
    buf = torch.full((R + 2, width if align else width + 1), fill, dtype=dtype, device="cuda")
    at = 32 if align else 3
    rows = buf[1:-1, at:at + C]
    if align:
        assert rows.data_ptr() % 32 == 0 and rows.stride(0) * rows.element_size() % 32 == 0
    return buf, rows


def untouched(buf, rows, fill):
    rows.fill_(fill)
    b = buf.float()
    return bool(torch.isnan(b).all() if fill != fill else (b == fill).all())


@pytest.mark.gpu
@pytest.mark.parametrize("align", [True, False])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("C", [16, 48, 100, 112, 128, 209, 512, 528, 640, 1025])
def test_every_output_leaves_what_lies_around_it(C, kind, t, align):
    """y, the 8-bit form, the restored y, dx, dw, db, the workspace and unpacked values, in rows of
    vectors (C a multiple of 16, align) where lanes exceed the row, and element by element."""
    R, nan = 37, float("nan")
    k, dt = T.norm._KINDS[kind]
    fill = 99 if kind == "int8" else 96  # 96 is an e4m3 number
    x, dy = (guarded(R, C, t, 0, align)[1].copy_(make(R, C, t, s)) for s in (C, C + 1))
    w = 1 + 0.3 * make(1, C, F32, C)[0]
    want_y, want_stats, want = T.norm_forward(x, w, checkpoint=kind)
    want_dx, want_dw, want_db = T.norm_backward(want, want_stats, dy, w)
    (yb, y), (cb, codes) = guarded(R, C, t, nan, align), guarded(R, C, dt, fill, align)
    eb, exps = guarded(R, (C + 31) // 32, torch.uint8, 77, align)
    stats = torch.full((2 * R + 8,), nan, device="cuda")
    Bd.tri_norm_fwd(x, w, None, y, stats[4:-4].view(2, R), codes, exps, k)
    assert torch.equal(y, want_y) and torch.equal(stats[4:-4].view(2, R), want_stats)
    assert torch.equal(codes.float(), want.codes.float()) and torch.equal(exps, want.exps)
    rb, again = guarded(R, C, t, nan, align)
    Bd.tri_norm_restore(codes, exps, k, want_stats, w, None, again)
    assert torch.equal(again, T.norm_restore(want, want_stats, w))
    ub, values = guarded(R, C, t, nan, align)
    Bd.tri_act8_unpack(codes, exps, k, values)
    assert torch.equal(values, T.act8_unpack(want))
    db_, dx = guarded(R, C, t, nan, align)
    need = Bd.tri_norm_bwd_workspace_bytes(R, C)
    ws = torch.full((need + 64,), 90, dtype=torch.uint8, device="cuda")
    sums = torch.full((2 * C + 12,), nan, device="cuda")
    dw, db = sums[4:C + 4], sums[C + 8:-4]
    Bd.tri_norm_bwd(None, codes, exps, k, want_stats, w, dy, dx, dw, db, ws[:need])
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw) and torch.equal(db, want_db)
    assert (ws[need:] == 90).all() and torch.isnan(sums[[0, 1, 2, 3, C + 4, C + 5, C + 6, C + 7, -4, -3, -2, -1]]).all()
    pb, codes2 = guarded(R, C, dt, fill, align)
    qb, exps2 = guarded(R, (C + 31) // 32, torch.uint8, 77, align)
    Bd.tri_act8_pack(x, codes2, exps2, k)
    assert torch.equal(codes2.float(), want.codes.float()) and torch.equal(exps2, want.exps)
    for buf, rows, f in ((yb, y, nan), (cb, codes, fill), (eb, exps, 77), (rb, again, nan), (ub, values, nan), (db_, dx, nan),
                         (pb, codes2, fill), (qb, exps2, 77)):
        assert untouched(buf, rows, f)
    assert torch.isnan(stats[:4]).all() and torch.isnan(stats[-4:]).all()


def test_eps_past_fp32_is_refused(lib):
    """Like an infinite one, with the library's own error."""
    x = torch.zeros(4, 8)
    for eps in (1e39, float("inf"), float("nan"), -1.0):
        for call in (lambda: T.norm_forward(x, eps=eps), lambda: T.layer_norm(x, eps=eps),
                     lambda: T.norm_linear(x, None, None, torch.zeros(3, 8), eps=eps)):
            with pytest.raises(Bd.TriAttnError) as e:
                call()
            assert e.value.status == Bd.TRI_ATTN_ERR_SHAPE
