"""The FP64 oracle of the norm, the 8-bit form and the relative position bias, pinned to closed
forms, torch and central differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import tri_norm_oracle as O


def test_norm_matches_torch_and_differences():
    g = np.random.default_rng(3)
    x, w, b, dy = g.normal(size=(5, 7)), g.normal(size=7), g.normal(size=7), g.normal(size=(5, 7))
    y, mean, rstd = O.fwd(x, w, b, 1e-5)
    t = torch.nn.functional.layer_norm(torch.tensor(x), (7,), torch.tensor(w), torch.tensor(b), 1e-5)
    np.testing.assert_allclose(y, t.numpy(), rtol=0, atol=1e-13)
    dx, dw, db = O.bwd(x, mean, rstd, w, dy)
    f = lambda x_, w_, b_: (O.fwd(x_, w_, b_, 1e-5)[0] * dy).sum()  # noqa: E731
    for k, (a, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        for i in np.ndindex(a.shape):
            d = np.zeros(a.shape)
            d[i] = 1e-5
            args = [[x, w, b], [x, w, b]]
            args[0][k], args[1][k] = a + d, a - d
            # central difference: h^2 f''' / 6 + rounding 1e-16 / h, both far below 1e-8
            assert abs((f(*args[0]) - f(*args[1])) / 2e-5 - grad[i]) < 1e-8


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_act8_definition(kind):
    x = np.zeros((6, 33))
    q = O.Q[kind]
    x[0, 0], x[1, 0], x[2, 0] = q, np.nextafter(np.float32(q), np.float32(1e9)), 1.0
    x[3, 5], x[4, 7], x[4, 32] = np.inf, np.nan, -3.0
    codes, exps, vals = O.act8(x, kind)
    assert exps[0, 0] == 127 and codes[0, 0] == q          # fits exactly
    assert exps[1, 0] == 128                               # just past: the next power of two
    assert 2 * np.abs(codes[2, 0]) > q and vals[2, 0] == 1.0
    assert exps[3, 0] == 255 and np.isnan(vals[3, :32]).all() and vals[3, 32] == 0
    assert exps[4, 0] == 255 and abs(vals[4, 32] + 3.0) <= 3.0 / 63
    assert exps[5, 0] == 1 and not vals[5].any()           # zeros: the least exponent


def test_e4m3_rounding_matches_torch():
    v = np.linspace(-448, 448, 20011)
    v = np.concatenate([v, v * 1e-3, v * 1e-5, [0.0, 2 ** -10, 3 * 2 ** -10, 2 ** -6]]).astype(np.float32)
    t = torch.tensor(v).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_round(v.astype(np.float64)), t)


def test_buckets_by_hand():
    edges = [-1, 0, 1, 2]  # distances <= -2, -1, 0, 1, >= 2
    pos = np.array([[0, 1, 5]], np.int32)
    np.testing.assert_array_equal(O.buckets(edges, pos, pos)[0], [[2, 3, 4], [1, 2, 4], [0, 0, 2]])
    grp = np.array([[0, 0, 1]], np.int32)
    np.testing.assert_array_equal(O.buckets(edges, pos, pos, grp, grp)[0], [[2, 3, 5], [1, 2, 5], [5, 5, 2]])
    far = np.array([[2 ** 31 - 1, -2 ** 31]], np.int32)  # differences past 32 bits
    np.testing.assert_array_equal(O.buckets(edges, far, far)[0], [[2, 0], [4, 2]])


def test_relpos_gradient_is_the_transpose():
    g = np.random.default_rng(5)
    pos = g.integers(-9, 9, (2, 6)).astype(np.int32)
    k = O.buckets([-2, 0, 3], pos, pos)
    table, d = g.normal(size=(4, 3)), g.normal(size=(2, 3, 6, 6))
    lhs = (O.relpos_fwd(table, k) * d).sum()
    assert abs(lhs - (table * O.relpos_bwd(d, k, 4)).sum()) < 1e-12
