"""The budgeted cache's 64-bit definitions (oracle/budget.py) against closed
forms and against counting by hand."""
import numpy as np
import pytest

from oracle import budget


def test_heads_have_unit_mean_square_and_keep_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64)) * 7
    for inter in (False, True):
        y, _ = budget.prepare_heads(x, np.zeros(64), 1.0, 0.0, np.array([0, 1, 5, 900, 10 ** 6]),
                                    1e4 ** (-np.arange(32) / 32), 64, inter)
        assert np.allclose((y * y).mean(-1), 1, atol=1e-12)


def test_rotation_is_relative_and_by_pairs():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 32))
    freq = 1e4 ** (-np.arange(8) / 8)

    def dot(a, b, inter):
        x, _ = budget.prepare_heads(q, None, 0, 0, np.array([a]), freq, 16, inter)
        y, _ = budget.prepare_heads(k, None, 0, 0, np.array([b]), freq, 16, inter)
        assert np.array_equal(x[..., 16:], q[..., 16:])
        return (x * y).sum()

    for inter in (False, True):
        assert np.isclose(dot(3, 10, inter), dot(1003, 1010, inter))
        assert not np.isclose(dot(3, 10, inter), dot(3, 11, inter))
    # one pair, a quarter turn: (a, b) -> (-b, a)
    x = np.zeros((1, 1, 32))
    x[..., 0], x[..., 8] = 2.0, 5.0
    y, size = budget.prepare_heads(x, None, 0, 0, np.array([1]), np.full(8, np.pi / 2), 16, False)
    assert np.allclose([y[0, 0, 0], y[0, 0, 8]], [-5, 2]) and size[0, 0, 0] == 7
    x[..., 1] = 3.0
    y, _ = budget.prepare_heads(x, None, 0, 0, np.array([1]), np.full(8, np.pi / 2), 16, True)
    assert np.allclose(y[0, 0, :2], [-3, 2])


def test_weights_of_a_step_add_up_to_its_queries():
    rng = np.random.default_rng(2)
    n, m, h, G, d = 4, 11, 2, 3, 16
    q, k = rng.standard_normal((n, h * G, d)), rng.standard_normal((m, h, d))
    seen = budget.visible(n, m)
    assert seen.sum() == sum(m - n + t + 1 for t in range(n))
    s = np.einsum("nhgd,mhd->nhgm", q.reshape(n, h, G, d), k) * 0.3
    s = np.where(seen[:, None, None], s, -np.inf)
    lse = np.log(np.exp(s).sum(-1)).reshape(n, h * G)
    w, loss = budget.key_weights(q, k, lse, seen, 0.3)
    assert np.allclose(w.sum(0), n * G) and np.all(loss > 0) and np.all(loss < 1e-3 * w + 1e-12)
    # a path: its queries alone, its keys in its order
    w2, _ = budget.key_weights(q, k, lse, seen, 0.3, path=[0, 2])
    assert w2.shape == (m - n + 2, h) and np.allclose(w2.sum(0) <= 2 * G, True)
    w0, _ = budget.key_weights(q[:1], k[:m - n + 1], lse[:1], seen[:1, :m - n + 1], 0.3)
    last, _ = budget.key_weights(q[2:3], k, lse[2:3], seen[2:3], 0.3)
    assert np.allclose(w2[:m - n], w0[:m - n] + last[:m - n]) and np.allclose(w2[-1], last[m - n + 2])
    # a query that saw nothing counts nothing
    lse[1] = -np.inf
    w3, _ = budget.key_weights(q, k, lse, seen, 0.3)
    assert np.allclose(w3.sum(0), (n - 1) * G)


def test_masks_by_bits():
    mask = np.array([0b10110101, 0b1], np.uint8)
    assert budget.visible(3, 5, mask).tolist() == [[True, True, True, False, True],
                                                   [True, True, False, True, True],
                                                   [True, True, False, True, True]]
    assert budget.visible(1, 4, mask, offset=4, full=True).tolist() == [[True, True, False, True]]


@pytest.mark.parametrize("w, keep, sinks, recent, want", [
    ([5, 1, 4, 2, 3], 2, 0, 0, [0, 2]), ([5, 1, 4, 2, 3], 3, 1, 1, [0, 2, 4]), ([1, 1, 1, 1], 2, 0, 0, [0, 1]),
    ([1, 2, 2, 2, 1], 2, 0, 1, [1, 4]), ([0.0, -0.0, 0.0], 2, 0, 0, [0, 1]), ([1, np.nan, 3], 1, 0, 0, [1]),
    ([np.inf, np.nan, -np.inf, 0], 3, 0, 0, [0, 1, 3]), ([1, 2, 3], 9, 1, 1, [0, 1, 2]), ([1, 2, 3, 4], 1, 2, 2, [0]),
    ([9, 1, 2, 3, 4, 8], 3, 2, 2, [0, 1, 5]), ([], 4, 1, 1, []), ([1, 2], 0, 1, 1, []),
])
def test_survivors(w, keep, sinks, recent, want):
    assert budget.survivors(np.array(w, np.float32), keep, sinks, recent) == want
