"""The branched-rollout oracle against independent statements (CPU)."""
import numpy as np
import pytest

from oracle import branch_oracle as O


def _rows(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dims", [(16,), (8, 4, 4), (4, 8), (16, 0)])
def test_rope_is_a_rotation_and_its_inverse_undoes_it(halves, dims):
    rng = np.random.default_rng(1)
    x, pos = _rows(rng, 3, 5, 24), rng.integers(-1000, 1000, (5, len(dims)))
    f = O.ladder(dims)
    y = O.rope(x, pos, dims, f, halves)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
    np.testing.assert_allclose(O.rope(y, pos, dims, f, halves, inverse=True), x, atol=1e-12)
    np.testing.assert_array_equal(y[..., sum(dims):], x[..., sum(dims):])


def test_rope_product_depends_on_the_distance_only():
    rng = np.random.default_rng(2)
    q, k, dims = _rows(rng, 1, 1, 16), _rows(rng, 1, 1, 16), (8, 4, 4)
    f = O.ladder(dims)
    at = lambda x, p: O.rope(x, np.array([p]), dims, f, False)[0, 0]  # noqa: E731
    a = at(q, (7, 3, 9)) @ at(k, (2, 1, 4))
    b = at(q, (107, 23, 59)) @ at(k, (102, 21, 54))
    assert abs(a - b) < 1e-11


def test_inverse_is_the_gradient_of_the_rotation():
    # d/dx of sum(w . rope(x)) is rope(w, inverse), here by central differences
    rng = np.random.default_rng(3)
    x, w, pos, dims = _rows(rng, 1, 2, 8), _rows(rng, 1, 2, 8), np.array([[3, 5], [11, 2]]), (4, 4)
    f = O.ladder(dims)
    g = O.rope(w, pos, dims, f, True, inverse=True)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-5
        num = ((O.rope(x + d, pos, dims, f, True) - O.rope(x - d, pos, dims, f, True)) * w).sum() / 2e-5
        assert abs(num - g[i]) < 1e-8


def _case(rng, H=2, g=2, D=8, page=4, length=(9, 0, 4), new=(3, 0, 4), C=6):
    B, most = len(length), 3
    table = rng.permutation(B * most + 2)[:B * most].reshape(B, most)
    K, V = _rows(rng, B * most + 2, H, page, D), _rows(rng, B * most + 2, H, page, D)
    cu = np.concatenate(([0], np.cumsum(new)))
    q = _rows(rng, H * g, cu[-1], D)
    return q, cu, K, V, table, np.array(length), (_rows(rng, H, C, D), _rows(rng, H, C, D))


def test_attention_equals_a_dense_softmax_with_repeated_keys():
    # a group of count m equals its key and value repeated m times (Lemma A.1)
    rng = np.random.default_rng(4)
    q, cu, K, V, table, length, (pK, pV) = _case(rng)
    m, size = rng.integers(1, 5, (2, 6)), np.array([6, 4])
    out, lse = O.branch_attention(q, cu, (pK, pV, m, size), K, V, table, length, 0.3)
    for e in range(4):
        h = e // 2
        for b in range(3):
            own = [(K[table[b, p // 4], h, p % 4], V[table[b, p // 4], h, p % 4]) for p in range(length[b])]
            rows = [(pK[h, j], pV[h, j]) for j in range(size[h]) for _ in range(m[h, j])] + own
            for t in range(cu[b], cu[b + 1]):
                x = np.array([0.3 * q[e, t] @ k for k, _ in rows])
                w = np.exp(x)
                np.testing.assert_allclose(out[e, t], sum(a * v for a, (_, v) in zip(w, rows)) / w.sum(), rtol=1e-10)
                np.testing.assert_allclose(lse[e, t], np.log(w.sum()), rtol=1e-10)


def test_a_hidden_group_and_rows_that_see_nothing():
    rng = np.random.default_rng(5)
    q, cu, K, V, table, length, (pK, pV) = _case(rng, new=(3, 0, 6), length=(9, 0, 4))
    gone = np.ones((2, 6), int)
    gone[:, 2] = 0
    a = O.branch_attention(q, cu, (pK, pV, gone, None), K, V, table, length, 0.3)[0]
    keep = [0, 1, 3, 4, 5]
    b = O.branch_attention(q, cu, (pK[:, keep], pV[:, keep], None, None), K, V, table, length, 0.3)[0]
    np.testing.assert_allclose(a, b, rtol=1e-12)
    # without a prefix the first two tokens of branch 2 (positions -2, -1) see nothing when causal
    out, lse = O.branch_attention(q, cu, None, K, V, table, length, 0.3, block=1)
    assert (out[:, cu[2]:cu[2] + 2] == 0).all() and np.isneginf(lse[:, cu[2]:cu[2] + 2]).all()
    assert np.isfinite(lse[:, cu[2] + 2:]).all()


def test_append_then_attend_equals_attention_over_the_concatenation():
    rng = np.random.default_rng(6)
    q, cu, K, V, table, length, _ = _case(rng)
    k, v = _rows(rng, 2, cu[-1], 8), _rows(rng, 2, cu[-1], 8)
    before = K.copy()
    O.page_append(K, V, k, v, cu, table, length)
    assert (K != before).any(axis=(1, 3)).sum() == cu[-1]
    out, _ = O.branch_attention(q, cu, None, K, V, table, length, 0.3, block=1)
    t = cu[1] - 1  # the last token of branch 0 sees all 9 positions
    x = np.array([0.3 * q[0, t] @ K[table[0, p // 4], 0, p % 4] for p in range(9)])
    w = np.exp(x) / np.exp(x).sum()
    np.testing.assert_allclose(out[0, t], sum(w[p] * V[table[0, p // 4], 0, p % 4] for p in range(9)), rtol=1e-10)
    np.testing.assert_array_equal(K[table[0, 2], :, 0], k[:, t])
