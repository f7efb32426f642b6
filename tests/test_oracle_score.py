"""The oracle of the biased and the differential attention against closed forms
and against differences, and the bucket helper (CPU)."""
import numpy as np
import pytest

from dynamic_block_sparse_fractal_b200 import api
from oracle import score

GRID = (2, 2, 4)  # 16 tokens: the oracle takes any grid
S = 16


def data(seed, d=8):
    rng = np.random.default_rng(seed)
    q, k, v, g = (rng.standard_normal((S, d)) for _ in range(4))
    keep = rng.random((S, S)) < 0.7
    keep[3] = False
    keep[:, 5] = False
    n = 2 * sum(GRID) - 3
    bucket = rng.integers(0, 7, n)
    return q, k, v, g, keep, bucket, rng.standard_normal(7)


def central(f, x, eps=1e-5):
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        out[i] = (f(a) - f(b)) / (2 * eps)
    return out


def test_bias_gradients_match_differences():
    q, k, v, g, keep, bucket, row = data(1)

    def loss(q=q, k=k, v=v, row=row):
        return (score.bias_head(q, k, v, keep, score.bias_matrix(row, bucket, *GRID))[0] * g).sum()

    O, P, lse = score.bias_head(q, k, v, keep, score.bias_matrix(row, bucket, *GRID))
    assert np.all(O[3] == 0) and lse[3] == -np.inf
    dq, dk, dv, dS = score.bias_head_backward(q, k, v, g, P, O)
    dt = score.bucket_sums(dS, bucket, 7, *GRID)
    # differences of step 1e-5: truncation 1e-10, rounding 2^-52 |loss| / 1e-5 < 1e-9
    for got, f, x in ((dq, lambda x: loss(q=x), q), (dk, lambda x: loss(k=x), k),
                      (dv, lambda x: loss(v=x), v), (dt, lambda x: loss(row=x), row)):
        np.testing.assert_allclose(got, central(f, x), atol=1e-7)


def test_diff_gradients_match_differences():
    q, k, v, g, keep, _, _ = data(2)
    lam = np.array([0.7])

    def loss(q=q, k=k, v=v, lam=lam):
        return (score.diff_head(q, k, v, keep, lam[0])[0] * g).sum()

    O, O2, P, lse = score.diff_head(q, k, v, keep, lam[0])
    dq, dk, dv, dl, _ = score.diff_head_backward(q, k, v, g, P, lam[0])
    for got, f, x in ((dq, lambda x: loss(q=x), q), (dk, lambda x: loss(k=x), k),
                      (dv, lambda x: loss(v=x), v), (np.array([dl]), lambda x: loss(lam=x), lam)):
        np.testing.assert_allclose(got, central(f, x), atol=1e-7)
    # equal maps: the difference is (1 - lambda) of one of them
    qq, kk = np.concatenate([q, q], 1), np.concatenate([k, k], 1)
    O, O2, _, _ = score.diff_head(qq, kk, np.concatenate([v, v], 1), keep, 0.25)
    np.testing.assert_allclose(O, 0.75 * O2, atol=1e-12)


def test_bias_of_one_axis_by_hand():
    # one row of four columns: offsets -3 .. 3 read entries 0 .. 6
    bucket = [0] + [0] + list(range(7))
    row = np.array([0.0, 1, 2, 3, 4, 5, 6])
    b = score.bias_matrix(row, bucket, 1, 1, 4)
    assert b[0].tolist() == [3, 4, 5, 6] and b[3].tolist() == [0, 1, 2, 3]
    row[6] = -3.4e38  # the lowest value masks
    assert score.bias_matrix(row, bucket, 1, 1, 4)[0, 3] == -np.inf


@pytest.mark.parametrize("n,b,far", [(1, 2, 1), (4, 8, 16), (33, 16, 32), (80, 24, 64)])
def test_relative_buckets(n, b, far):
    m, count = api.relative_buckets(n, 1, 1, (b, 2, 2), (far, 1, 1), device="cpu")
    m = m.numpy()
    assert count == b + 4 and m.shape == (2 * n - 1 + 2,)
    t = m[:2 * n - 1]
    assert t.min() >= 0 and t.max() < b
    near, pos = t[:n][::-1], t[n - 1:]  # offsets 0, -1, ..; 0, 1, ..
    assert near[0] == 0 and np.all(np.diff(near) >= 0)
    assert np.array_equal(pos[1:], near[1:] + b // 2)  # the signs have buckets of their own
    exact = max(1, b // 4)
    assert near[:exact].tolist() == list(range(min(n, exact)))
    assert m[2 * n - 1] == b and m[2 * n] == b + 2  # the other axes' own buckets
    with pytest.raises(ValueError):
        api.relative_buckets(4, 4, 4, (3, 4, 4), device="cpu")
