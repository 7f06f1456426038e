"""The learned relative position bias (tri_relpos_fwd, tri_relpos_bwd): host-side checks (no
GPU) and GPU parity against the FP64 oracle (oracle/tri_norm_oracle.py)."""
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
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return Bd.load()


def test_struct_layout_matches_the_header():
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "tri_attn.h"
int main(void){
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(tri_relpos_fwd_args), offsetof(tri_relpos_fwd_args, table),
         offsetof(tri_relpos_fwd_args, base), sizeof(tri_relpos_bwd_args), offsetof(tri_relpos_bwd_args, dtable),
         offsetof(tri_relpos_bwd_args, workspace_bytes));
  return 0; }
'''
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    F, W = Bd.RelposFwdArgs, Bd.RelposBwdArgs
    assert got == [ctypes.sizeof(F), F.table.offset, F.base.offset, ctypes.sizeof(W), W.dtable.offset,
                   W.workspace_bytes.offset]


def fake():
    """Aligned but fake pointers: every case is rejected before anything could use them."""
    a = Bd.RelposBwdArgs()
    f = a.f
    f.B, f.H, f.Nq, f.Nk, f.E = 2, 4, 64, 72, 64
    f.table, f.edges, f.pos_q, f.pos_k, f.group_q, f.group_k = (0x10000 + k * 0x1000000 for k in range(6))
    f.q_stride, f.k_stride = 64, 72
    for k, t in enumerate((f.base, f.bias, a.dbias)):
        t.ptr = 0x9000000 + k * 0x1000000
        for x, s in enumerate((4 * 64 * 72, 64 * 72, 72, 1)):
            t.stride[x] = s
    a.dtable, a.workspace = 0xD000000, 0xE000000
    a.workspace_bytes = Bd.tri_relpos_bwd_workspace_bytes(2, 4, 64, 72, 64, True)
    return a


FWD_REFUSALS = [
    ({"B": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"H": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"Nq": 0}, Bd.TRI_ATTN_ERR_SHAPE),
    ({"Nk": -8}, Bd.TRI_ATTN_ERR_SHAPE), ({"B": 1, "Nk": 8, "Nq": 2 ** 30 + 1}, Bd.TRI_ATTN_ERR_SHAPE),
    ({"B": 1, "Nq": 1, "Nk": 2 ** 30 + 1}, Bd.TRI_ATTN_ERR_SHAPE), ({"E": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"E": 511}, Bd.TRI_ATTN_ERR_UNSUPPORTED),
    ({"H": 4097}, Bd.TRI_ATTN_ERR_UNSUPPORTED), ({"B": 2 ** 20, "Nq": 2 ** 11}, Bd.TRI_ATTN_ERR_SHAPE),
    ({"edges": None}, Bd.TRI_ATTN_ERR_NULL), ({"pos_q": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"group_k": None}, Bd.TRI_ATTN_ERR_NULL), ({"table": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"table_type": 3}, Bd.TRI_ATTN_ERR_DTYPE), ({"q_stride": -64}, Bd.TRI_ATTN_ERR_STRIDE),
    ({"pos_k": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN), ({"table": 0x10001}, Bd.TRI_ATTN_ERR_ALIGN),
    ({"bias__ptr": None}, Bd.TRI_ATTN_ERR_NULL), ({"bias__ptr": 0x10008}, Bd.TRI_ATTN_ERR_ALIGN),
    ({"bias__stride__2": 76}, Bd.TRI_ATTN_ERR_STRIDE), ({"bias__stride__2": 64}, Bd.TRI_ATTN_ERR_STRIDE),
    ({"bias__stride__1": 0}, Bd.TRI_ATTN_ERR_STRIDE), ({"base__stride__3": 2}, Bd.TRI_ATTN_ERR_STRIDE),
]
BWD_REFUSALS = [
    ({"f__E": 0}, Bd.TRI_ATTN_ERR_SHAPE), ({"f__pos_k": None}, Bd.TRI_ATTN_ERR_NULL), ({"dbias__ptr": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"dbias__stride__0": 4}, Bd.TRI_ATTN_ERR_STRIDE), ({"dtable": None}, Bd.TRI_ATTN_ERR_NULL),
    ({"dtable": 0x10002}, Bd.TRI_ATTN_ERR_ALIGN), ({"workspace": None}, Bd.TRI_ATTN_ERR_WORKSPACE),
    ({"workspace_bytes": 100}, Bd.TRI_ATTN_ERR_WORKSPACE), ({"workspace": 0x10004}, Bd.TRI_ATTN_ERR_ALIGN),
]


def change(a, what):
    for k, v in what.items():
        obj, names = a, k.split("__")
        for n in names[:-1]:
            obj = getattr(obj, n)
        if names[-1].isdigit():
            obj[int(names[-1])] = v
        else:
            setattr(obj, names[-1], v)
    return bytes(a)


@pytest.mark.parametrize("what,want", FWD_REFUSALS)
def test_fwd_refusals(lib, what, want):
    assert lib.tri_relpos_fwd(change(fake().f, what), None) == want


@pytest.mark.parametrize("what,want", BWD_REFUSALS)
def test_bwd_refusals(lib, what, want):
    assert lib.tri_relpos_bwd(change(fake(), what), None) == want


def test_workspace_bytes(lib):
    ws = Bd.tri_relpos_bwd_workspace_bytes
    assert lib.tri_relpos_fwd(None, None) == lib.tri_relpos_bwd(None, None) == Bd.TRI_ATTN_ERR_NULL
    assert ws(1, 4, 64, 64, 0, False) == ws(1, 0, 64, 64, 8, False) == ws(0, 4, 64, 64, 8, False) == 0
    for B, H, N, E in ((1, 4, 768, 64), (2, 12, 1031, 39), (1, 1, 1, 1), (1, 40, 2048, 510), (3, 4096, 5, 510)):
        assert 0 < ws(B, H, N, N, E, False) <= ws(B, H, N, N, E, True) <= 148 * 8 * (E + 2) * H * 4


def test_edges_helpers():
    assert T.relpos_edges_clipped(2, "cpu").tolist() == [-1, 0, 1, 2]
    assert T.relpos_edges_log(4, 16, "cpu").tolist() == [-15, -5, -1, 0, 1, 2, 6, 16]  # 2 * 8^(1/2) -> 6, 2 * 8 -> 16
    for per, far in ((1, 1), (3, 3), (16, 128), (20, 200000), (255, 255), (255, 2 ** 31 - 1)):
        e = T.relpos_edges_log(per, far, "cpu").tolist()
        assert e == sorted(set(e)) and len(e) == 2 * per and [1 - x for x in reversed(e)] == e
    for bad in (lambda: T.relpos_edges_clipped(0, "cpu"), lambda: T.relpos_edges_clipped(256, "cpu"),
                lambda: T.relpos_edges_log(8, 7, "cpu"), lambda: T.relpos_edges_log(8, 2 ** 31, "cpu")):
        with pytest.raises(Bd.TriAttnError):
            bad()


def test_python_refusals_on_cpu(lib):
    pos, e = torch.arange(8, dtype=I32), T.relpos_edges_clipped(3, "cpu")
    t = torch.zeros(7, 4)
    with pytest.raises(Bd.TriAttnError, match="CUDA device"):
        T.relpos_forward(t, e, pos, pos)
    for args, want in (((t[:6], e, pos, pos), Bd.TRI_ATTN_ERR_SHAPE), ((t, e, pos.long(), pos), Bd.TRI_ATTN_ERR_DTYPE),
                       ((t, e.long(), pos, pos), Bd.TRI_ATTN_ERR_DTYPE), ((t.half(), e, pos, pos), Bd.TRI_ATTN_ERR_DTYPE),
                       ((t[0], e, pos, pos), Bd.TRI_ATTN_ERR_SHAPE), ((t, e, pos, pos, None, None, t), Bd.TRI_ATTN_ERR_SHAPE),
                       ((t, e, torch.zeros(2, 8, dtype=I32), torch.zeros(3, 8, dtype=I32)), Bd.TRI_ATTN_ERR_SHAPE),
                       ((t, e, pos, pos, pos, pos), Bd.TRI_ATTN_ERR_SHAPE), ((t, e, pos, pos, pos), Bd.TRI_ATTN_ERR_NULL),
                       ((t, e, pos, pos, None, None, torch.zeros(1, 4, 8, 16, dtype=BF)), Bd.TRI_ATTN_ERR_SHAPE)):
        with pytest.raises(Bd.TriAttnError) as err:
            T.relpos_forward(*args)
        assert err.value.status == want
    for d in (torch.zeros(1, 4, 8, 9, dtype=BF), torch.zeros(4, 8, 8, dtype=BF)):
        with pytest.raises(Bd.TriAttnError) as err:
            T.relpos_backward(d, e, pos, pos)
        assert err.value.status == Bd.TRI_ATTN_ERR_SHAPE


def test_a_bias_of_another_dtype_is_refused_and_not_cast(lib):
    pos, e = torch.arange(9, dtype=I32), T.relpos_edges_clipped(3, "cpu")
    for n in (8, 9):
        d = torch.zeros(1, 4, n, n)
        for call in (lambda: T.relpos_backward(d, e, pos[:n], pos[:n]),
                     lambda: T.relpos_forward(torch.zeros(7, 4), e, pos[:n], pos[:n], base=d)):
            with pytest.raises(Bd.TriAttnError) as err:
                call()
            assert err.value.status == Bd.TRI_ATTN_ERR_DTYPE


def test_rows_that_end_with_their_storage_are_copied():
    """Odd rows whose last 16 bytes reach past the storage are not handed to the kernels as they are."""
    full = torch.zeros(2 * 16, dtype=BF)
    view = full.as_strided((1, 1, 2, 13), (32, 32, 16, 1))
    assert T.relpos._layout(view).data_ptr() == view.data_ptr()
    short = torch.empty(16 + 13, dtype=BF).as_strided((1, 1, 2, 13), (32, 32, 16, 1))
    if short.data_ptr() % 16 == 0:
        assert T.relpos._layout(short).data_ptr() != short.data_ptr()
    assert T.relpos._layout(full.as_strided((1, 1, 2, 16), (32, 32, 16, 1))).data_ptr() == full.data_ptr()
    odd = torch.zeros(1, 1, 4, 13, dtype=BF)  # rows at odd elements
    assert T.relpos._layout(odd).stride(2) == 16


# ---------------------------------------------------------------------------
# GPU parity
# ---------------------------------------------------------------------------
EDGES = {
    "clip": list(range(-31, 33)), "one": [0], "twice": [-3, -3, 0, 0, 5], "far": [-200000, -9000, -40, 0, 1, 41, 9001, 200001],
    "many": list(range(-254, 256)), "span": [-1000, 1046], "wide": [-1000, 1047],  # the last two: just within and past the lookup
    "ends": [-2 ** 31 + 1, -5, 6, 2 ** 31 - 1],
}
CASES = [  # B, H, Nq, Nk, edges, groups, base, table type
    (1, 4, 1, 1, "clip", 0, False, F32), (1, 4, 32, 32, "clip", 0, False, F32), (2, 4, 33, 40, "clip", 3, True, F32),
    (1, 1, 100, 257, "clip", 2, False, BF), (1, 3, 50, 71, "one", 0, True, F32), (2, 5, 17, 9, "twice", 2, False, F32),
    (1, 16, 1, 700, "far", 0, False, F32), (1, 17, 40, 64, "clip", 2, True, BF), (1, 33, 20, 31, "clip", 0, False, F32),
    (1, 2, 300, 301, "many", 2, True, F32), (1, 40, 24, 24, "many", 2, False, F32), (3, 8, 29, 200, "span", 0, False, F32),
    (3, 8, 29, 200, "wide", 0, False, F32), (1, 4, 60, 60, "ends", 0, False, F32), (1, 32, 70, 130, "far", 5, True, F32),
    (1, 12, 515, 515, "clip", 4, False, F32),
]


def make(B, H, Nq, Nk, edges, groups, base, tt, seed=0):
    g = np.random.default_rng(seed + 1000 * Nq + Nk)
    e = EDGES[edges]
    if edges == "ends":
        pos = [g.choice([-2 ** 31, 2 ** 31 - 1, 0, 7, -2 ** 31 + 3, 2 ** 31 - 9], (B, n)) for n in (Nq, Nk)]
    else:  # ascending runs with gaps, and in every second batch in no order
        pos = [np.cumsum(1 + 400 * (g.random((B, n)) < 0.05), 1) for n in (Nq, Nk)]
        for p in pos:
            p[1::2] = g.permuted(p[1::2], axis=1) * 31 - 3000
    pq, pk = (torch.tensor(p, dtype=I32).cuda() for p in pos)
    gq = gk = None
    if groups:
        gq, gk = (torch.tensor(np.sort(g.integers(0, groups, (B, n)), 1), dtype=I32).cuda() for n in (Nq, Nk))
    nb = len(e) + 1 + bool(groups)
    table = torch.tensor(g.normal(size=(nb, H)), dtype=F32).to(tt).cuda()
    pad = (Nk + 7) // 8 * 8 + 8
    full = lambda: torch.tensor(g.normal(size=(B, H, Nq, pad)), dtype=F32).to(BF).cuda()[..., :Nk]  # noqa: E731
    return table, torch.tensor(e, dtype=I32).cuda(), pq, pk, gq, gk, full() if base else None, full()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def bucket_of(e, pq, pk, gq, gk):
    n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return O.buckets(e.tolist(), n(pq), n(pk), n(gq), n(gk))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_parity(case):
    table, e, pq, pk, gq, gk, base, d = make(*case)
    k = bucket_of(e, pq, pk, gq, gk)
    bias = T.relpos_forward(table, e, pq, pk, gq, gk, base)
    assert bias.dtype == BF and all(s % 8 == 0 for s in bias.stride()[:3])
    ref = O.relpos_fwd(f64(table), k, f64(base))
    if base is None:
        assert torch.equal(bias.float().cpu(), torch.tensor(ref).float().to(BF).float())  # one rounding of the table
    else:  # one FP32 sum, one rounding to BF16
        err = np.abs(f64(bias) - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + U * (np.abs(ref) + np.abs(f64(base))))
    dt = T.relpos_backward(d, e, pq, pk, gq, gk)
    assert dt.dtype == F32 and dt.shape == table.shape
    D = f64(d)
    # a lane adds the rows of its task (< 515) to one register, eight values at a time in three
    # steps, or value by value into its word (< 8 x 515); then < 64 + 32 + 32 partial sums
    tol = (8 * 515 + 131) * U * O.relpos_bwd(np.abs(D), k, table.shape[0])
    assert np.all(np.abs(f64(dt) - O.relpos_bwd(D, k, table.shape[0])) <= tol)
    assert torch.equal(dt, T.relpos_backward(d, e, pq, pk, gq, gk))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 20, 41, 64, 71, 130])
@pytest.mark.parametrize("H", [1, 2, 5, 8, 33])
def test_small_whole_numbers_are_summed_exactly(N, H):
    """One block and many, every split of heads: sums of small whole numbers are exact."""
    g = torch.Generator().manual_seed(N * 40 + H)
    pos = torch.cumsum(1 + (torch.rand(N, generator=g) < 0.2).int() * 3, 0).int().cuda()
    d = torch.randint(-8, 9, (1, H, N, (N + 7) // 8 * 8), generator=g).to(BF).cuda()[..., :N]
    for e in (T.relpos_edges_clipped(4), T.relpos_edges_log(6, 5000)):
        k = bucket_of(e, pos[None], pos[None], None, None)
        np.testing.assert_array_equal(f64(T.relpos_backward(d, e, pos, pos)), O.relpos_bwd(f64(d), k, e.numel() + 1))


@pytest.mark.gpu
def test_exact_sums_and_broadcast_gradients():
    """Small whole numbers are added without rounding: every sum is exact."""
    table, e, pq, pk, gq, gk, _, d = make(2, 4, 190, 203, "clip", 3, False, F32)
    d = torch.randint(-8, 9, d.shape, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    k = bucket_of(e, pq, pk, gq, gk)
    want = O.relpos_bwd(f64(d), k, table.shape[0])
    np.testing.assert_array_equal(f64(T.relpos_backward(d, e, pq, pk, gq, gk)), want)  # unpadded rows: copied
    one = torch.ones((), dtype=BF, device="cuda").expand(d.shape)  # every stride 0
    want = np.repeat(np.bincount(k.ravel(), minlength=table.shape[0])[:, None], 4, 1)
    np.testing.assert_array_equal(f64(T.relpos_backward(one, e, pq, pk, gq, gk)), want)
    # gradient rows shared by the queries (stride 0), padded keys
    row = torch.randint(-8, 9, (2, 4, 1, 208), generator=torch.Generator().manual_seed(2)).to(BF).cuda()[..., :203]
    got = T.relpos_backward(row.expand(2, 4, 190, 203), e, pq, pk, gq, gk)
    want = O.relpos_bwd(f64(row.expand(2, 4, 190, 203)), k, table.shape[0])
    np.testing.assert_array_equal(f64(got), want)


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_bucket():
    table, e, pq, pk, gq, gk, _, d = make(1, 4, 64, 96, "clip", 0, False, F32)
    k = bucket_of(e, pq, pk, gq, gk)[0]
    d[0, 1, 10, 11] = float("nan")
    d[0, 2, 60, 3] = float("inf")
    dt = T.relpos_backward(d, e, pq, pk)
    bad = torch.zeros_like(dt, dtype=torch.bool)
    bad[k[10, 11], 1] = bad[k[60, 3], 2] = True
    assert torch.equal(~torch.isfinite(dt), bad)
    table[5, 0] = float("-inf")  # a bucket that is masked out
    table[6, 1] = torch.finfo(F32).min
    bias = T.relpos_forward(table, e, pq, pk)
    ref = table.to(BF)[torch.tensor(k).cuda()].permute(2, 0, 1)[None]
    assert torch.equal(bias, ref)


@pytest.mark.gpu
def test_shared_positions_and_layouts():
    table, e, pq, pk, gq, gk, base, d = make(2, 4, 40, 40, "clip", 2, True, F32)
    # positions [N] for the whole batch, groups per batch
    got = T.relpos_forward(table, e, pk[0], pk[0], gk, gk, base)
    want = T.relpos_forward(table, e, pk[:1].repeat(2, 1), pk[:1].repeat(2, 1), gk, gk, base)
    assert torch.equal(got, want)
    got = T.relpos_backward(d, e, pk[0], pk[0], gk[0], gk[0])
    want = T.relpos_backward(d, e, pk[:1].repeat(2, 1), pk[:1].repeat(2, 1), gk[:1].repeat(2, 1), gk[:1].repeat(2, 1))
    assert torch.equal(got, want)
    # every second position of a longer list; a base in another order of dimensions
    long = torch.stack([pk, pk + 1], -1).flatten(1)
    got = T.relpos_forward(table, e, long[:, ::2], pk, gk, gk, base.permute(0, 2, 3, 1).contiguous().permute(0, 3, 1, 2))
    assert torch.equal(got, T.relpos_forward(table, e, pk, pk, gk, gk, base))
    # a bias whose heads lie between its rows, and nothing written past Nk
    out = torch.full((2, 40, 4, 48), float("nan"), dtype=BF, device="cuda")
    Bd.tri_relpos_fwd(table, e, pk, pk, gk, gk, base, out.transpose(1, 2)[..., :40])
    assert torch.equal(out.transpose(1, 2)[..., :40], got) and torch.isnan(out[..., 40:]).all()
    table, e, pq, pk, *_ = make(1, 4, 5, 13, "clip", 0, False, F32)
    out = torch.full((1, 4, 5, 16), float("nan"), dtype=BF, device="cuda")
    Bd.tri_relpos_fwd(table, e, pq, pk, None, None, None, out[..., :13])
    assert torch.isfinite(out[..., :13]).all() and torch.isnan(out[..., 13:]).all()


@pytest.mark.gpu
def test_large_bias_past_32_bits():
    """Element offsets past 2^31: the last row equals the same row computed alone."""
    H, N = 16, 12000
    pos = torch.arange(N, dtype=I32, device="cuda")
    e = T.relpos_edges_clipped(32)
    table = torch.randn(65, H, generator=torch.Generator().manual_seed(0)).cuda()
    bias = T.relpos_forward(table, e, pos, pos)
    assert bias.numel() > 2 ** 31
    for rows in (slice(0, 1), slice(N - 1, N)):
        assert torch.equal(bias[:, :, rows], T.relpos_forward(table, e, pos[rows], pos))
    dt = T.relpos_backward(bias, e, pos, pos)
    # the table's rows were rounded once to BF16; each bucket holds that value so many times
    counts = torch.tensor([N - abs(x) for x in range(-32, 33)], dtype=torch.float64)
    counts[0] = counts[-1] = (N - 32) * (N - 31) / 2
    want = table.to(BF).double().cpu() * counts[:, None]
    # equal terms of one sign: a lane adds < 12000 x 8 / 8 eights, at most half a step each
    assert ((dt.double().cpu() - want).abs() <= 12400 * U * want.abs()).all()


@pytest.mark.gpu
def test_autograd():
    """The table's and the base's gradients, also against differences of the formula (linear: exact)."""
    table, e, pq, pk, gq, gk, base, up = make(2, 4, 21, 21, "clip", 2, True, F32)
    k = bucket_of(e, pk, pk, gk, gk)
    t, b = table.clone().requires_grad_(), base.clone().requires_grad_()
    bias = T.relative_position_bias(t, e, pk, group_q=gk, base=b)
    assert torch.equal(bias, T.relpos_forward(table, e, pk, pk, gk, gk, base))
    bias.backward(up)
    assert torch.equal(b.grad, up)
    want = O.relpos_bwd(f64(up), k, table.shape[0])
    assert np.all(np.abs(f64(t.grad) - want) <= 300 * U * O.relpos_bwd(np.abs(f64(up)), k, table.shape[0]))
    one = np.zeros(table.shape)
    one[3, 2] = 1.0
    diff = ((O.relpos_fwd(f64(table) + one, k) - O.relpos_fwd(f64(table) - one, k)) * f64(up)).sum() / 2
    assert abs(diff - t.grad[3, 2].item()) <= 300 * U * np.abs(f64(up)).sum() + 1e-9
    tb = table.to(BF).requires_grad_()
    T.relative_position_bias(tb, e, pk, group_q=gk).sum().backward()  # a gradient of stride 0
    assert tb.grad.dtype == BF and tb.grad.shape == table.shape


@pytest.mark.gpu
def test_streams_and_graphs():
    table, e, pq, pk, gq, gk, base, d = make(2, 4, 130, 131, "clip", 3, True, F32)
    run = lambda: (T.relpos_forward(table, e, pq, pk, gq, gk, base), T.relpos_backward(d, e, pq, pk, gq, gk))  # noqa: E731
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    table.mul_(2)
    pk.add_(3)
    d.mul_(-1)
    want = run()
    for g, out in graphs + graphs:
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_pending_device_error_stops_the_bias_too():
    table, e, pq, pk, gq, gk, base, d = make(1, 4, 32, 32, "clip", 0, False, F32)
    out = torch.full((1, 4, 32, 32), float("nan"), dtype=BF, device="cuda")
    dt = torch.full_like(table, float("nan"))
    ws = torch.empty(Bd.tri_relpos_bwd_workspace_bytes(1, 4, 32, 32, 64, False), dtype=torch.uint8, device="cuda")
    Bd.tri_attn_set_wait_limit_ns(1_000_000)
    try:
        Bd.tri_attn_selftest_expire_wait()
        Bd.tri_relpos_fwd(table, e, pq, pk, None, None, None, out)
        Bd.tri_relpos_bwd(d, e, pq, pk, None, None, dt, ws)
        torch.cuda.synchronize()
        assert torch.isnan(out).all() and torch.isnan(dt).all()
    finally:
        Bd.tri_attn_set_wait_limit_ns(2_000_000_000)
        Bd.tri_attn_device_error(True)


def test_log_edges_reach_the_distance_asked_for():
    """The last bucket of a side starts at max_distance, for every number of buckets."""
    pairs = [(1, 1), (1, 2), (1, 100), (1, 2 ** 31 - 1), (2, 2), (2, 7), (3, 3), (16, 128), (20, 200000), (255, 255),
             (255, 2 ** 31 - 1)]
    pairs += [(per, far) for per in range(1, 41) for far in range(per, 90, 7)]
    for per, far in pairs:
        e = T.relpos_edges_log(per, far, "cpu").tolist()
        assert e[-1] == far and e == sorted(set(e)) and len(e) == 2 * per and [1 - x for x in reversed(e)] == e
        if per > 1:  # distance 0 has a bucket of its own
            assert 0 in e and 1 in e
    assert T.relpos_edges_log(1, 100, "cpu").tolist() == [-99, 100]


def test_groups_of_their_own_over_shared_positions(monkeypatch):
    """Without pos_k the keys have the queries' positions, but the groups that were given for them."""
    seen = []
    monkeypatch.setattr(T.relpos, "relpos_forward", lambda *a: seen.append(a) or torch.zeros(1, 4, 8, 8, dtype=BF))
    pos, e, t = torch.arange(8, dtype=I32), T.relpos_edges_clipped(3, "cpu"), torch.zeros(8, 4)
    gq, gk = pos // 4, pos // 2
    for kw, want in (({}, (None, None)), ({"group_q": gq}, (gq, gq)), ({"group_q": gq, "group_k": gk}, (gq, gk)),
                     ({"group_k": gk}, (None, gk)), ({"pos_k": pos, "group_q": gq}, (gq, None))):
        T.relative_position_bias(t, e, pos, **kw)
        _, _, pq, pk, got_q, got_k, _ = seen.pop()
        assert pq is pos and pk is pos and got_q is want[0] and got_k is want[1]


@pytest.mark.gpu
def test_groups_of_their_own_over_shared_positions_on_the_gpu():
    table, e, _, pk, _, gk, base, d = make(2, 4, 40, 40, "clip", 3, True, F32)
    gq = gk.flip(1).contiguous()
    t = table.clone().requires_grad_()
    bias = T.relative_position_bias(t, e, pk, group_q=gq, group_k=gk, base=base)
    assert torch.equal(bias, T.relpos_forward(table, e, pk, pk, gq, gk, base))
    assert not torch.equal(bias, T.relpos_forward(table, e, pk, pk, gq, gq, base))
    bias.backward(d)
    assert torch.equal(t.grad, T.relpos_backward(d, e, pk, pk, gq, gk))
    for kw in ({"group_k": gk}, {"pos_k": pk, "group_q": gq}):  # one of the two alone
        with pytest.raises(Bd.TriAttnError) as err:
            T.relative_position_bias(table, e, pk, **kw)
        assert err.value.status == Bd.TRI_ATTN_ERR_NULL


@pytest.mark.parametrize("N", [8, 9, 21])
def test_the_bias_can_be_changed_in_place(monkeypatch, N):
    """Odd rows lie in a padded buffer of which the result must not be a view for autograd, which
    refuses in-place changes of a view made within a Function."""
    def forward(table, e, q, k, gq, gk, base, bias):
        bias.copy_(table[0, :, None, None].expand(bias.shape))

    monkeypatch.setattr(Bd, "tri_relpos_fwd", forward)
    e, pos = T.relpos_edges_clipped(3, "cpu"), torch.arange(N, dtype=I32)
    t = torch.ones(7, 4).requires_grad_()
    bias = T.relative_position_bias(t, e, pos)
    pad = (N + 7) // 8 * 8
    assert bias.shape == (1, 4, N, N) and bias.stride()[1:] == (N * pad, pad, 1)
    assert bias.untyped_storage().nbytes() >= 2 * 4 * N * pad  # the last row's last 16 bytes exist
    other = torch.full((), 2.0, dtype=BF).requires_grad_()
    bias += other
    assert bias.requires_grad and (bias == 3).all()
    bias.masked_fill_(pos[None, :] > 5, -1e9)
    monkeypatch.setattr(T.relpos, "relpos_backward", lambda g, *a: g.float().sum((0, 2, 3))[None].expand(7, 4))
    bias.sum().backward()
    assert (t.grad == 6 * N).all() and other.grad == 24 * N  # six keys of each row are left, four heads
    assert bias.detach().stride() == bias.stride()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [40, 41])
def test_the_bias_can_be_changed_in_place_on_the_gpu(N):
    table, e, _, pk, *_, base, d = make(2, 4, N, N, "clip", 0, True, F32)
    t = table.clone().requires_grad_()
    bias = T.relative_position_bias(t, e, pk)
    assert T.relpos._layout(bias).data_ptr() == bias.data_ptr()  # the layout that the kernels read
    want = bias.detach() + base
    bias += base
    assert torch.equal(bias, want)
    bias.backward(d)
    assert torch.equal(t.grad, T.relpos_backward(d, e, pk, pk))


def test_the_backward_launches_no_more_blocks_than_run_at_once(lib):
    """Every block costs its zeroed columns, its look-up table and a partial sum.  A block's shared
    memory (8 warps x buckets x 128 bytes + 6 KB, + 1 KB of its own) fits twice into an SM's 228 KB
    up to 107 buckets."""
    for E, per_sm in ((64, 2), (106, 2), (107, 1), (190, 1), (300, 1), (510, 1)):
        for H, N in ((4, 768), (16, 2048), (1, 4096)):
            heads = -(-H // 4) if H >= 4 else 1  # blocks of heads, each with its own columns
            blocks = Bd.tri_relpos_bwd_workspace_bytes(1, H, N, N, E, False) // ((E + 1) * H * 4)
            assert 0 < blocks <= 148 * per_sm, (E, H, N, blocks)
            # the rows are cut for the warps that run at once, over all blocks of heads, each of which
            # may end in a block that is not full
            assert blocks * heads <= 148 * per_sm + heads, (E, H, N, blocks)


def test_edges_of_another_shape_are_refused_in_both_directions(lib):
    pos, t, d = torch.arange(8, dtype=I32), torch.zeros(7, 4), torch.zeros(1, 4, 8, 8, dtype=BF)
    for e in (torch.tensor(3, dtype=I32), torch.zeros(2, 3, dtype=I32)):
        for call in (lambda: T.relpos_forward(t, e, pos, pos), lambda: T.relpos_backward(d, e, pos, pos)):
            with pytest.raises(Bd.TriAttnError) as err:
                call()
            assert err.value.status == Bd.TRI_ATTN_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("r", [52, 53, 54, 96, 97, 128, 255])
@pytest.mark.parametrize("B,H,N", [(1, 4, 771), (2, 12, 300)])
def test_many_buckets_are_summed_exactly(B, H, N, r):
    """Tables around the sizes at which an SM holds one block in place of two, and a block fewer
    warps (107 and 194 buckets): sums of small whole numbers are exact."""
    g = torch.Generator().manual_seed(r * N)
    pos = torch.cumsum(1 + (torch.rand(N, generator=g) < 0.1).int() * 40, 0).int()
    grp = (torch.arange(N) * 3 // N).int()
    d = torch.randint(-8, 9, (B, H, N, (N + 7) // 8 * 8), generator=g).to(BF)[..., :N]
    k = ((pos[None] - pos[:, None]).clamp(-r, r) + r).numpy()
    for gq in (None, grp):
        kk = k if gq is None else np.where(grp[:, None] == grp[None], k, 2 * r + 1)
        kk = np.broadcast_to(kk, (B, N, N))
        cu = lambda t: None if t is None else t.cuda()  # noqa: E731
        got = T.relpos_backward(d.cuda(), T.relpos_edges_clipped(r), cu(pos), cu(pos), cu(gq), cu(gq))
        np.testing.assert_array_equal(f64(got), O.relpos_bwd(f64(d), kk, 2 * r + 1 + (gq is not None)))
