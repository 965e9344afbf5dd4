"""The fp64 oracle of the token-by-token operators (oracle/token.py) on hand
values and invariants."""
import numpy as np
import pytest

import oracle


def test_rotation_by_hand():
    # one pair, quarter turn: (u, v) -> (-v, u)
    y = oracle.norm_rotate([3.0, 4.0], 1, None, 0.0, [np.pi / 2], False)
    np.testing.assert_allclose(y, [-4.0, 3.0], atol=1e-15)
    # split pairs (0, 2), (1, 3); the tail is left alone
    y = oracle.norm_rotate([1, 2, 3, 4, 5], 1, None, 0.0, [np.pi, 0.0], False)
    np.testing.assert_allclose(y, [-1, 2, -3, 4, 5], atol=1e-15)
    # interleaved pairs (0, 1), (2, 3)
    y = oracle.norm_rotate([1, 2, 3, 4, 5], 1, None, 0.0, [np.pi, 0.0], True)
    np.testing.assert_allclose(y, [-1, -2, 3, 4, 5], atol=1e-15)


def test_norm_gives_unit_mean_square_and_rotation_keeps_it():
    rng = np.random.default_rng(3)
    x = rng.normal(size=64)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    for inter in (False, True):
        y = oracle.norm_rotate(x, 12345, np.ones(64), 0.0, f, inter)
        assert abs(np.mean(y * y) - 1.0) < 1e-13
    # scores depend on the distance of two positions only
    a = [oracle.norm_rotate(x, p, None, 0.0, f, False) for p in (10, 17, 1010, 1017)]
    assert abs(a[0] @ a[1] - a[2] @ a[3]) < 1e-10


def test_decode_attention_is_the_oracles_dense_attention_of_one_row():
    rng = np.random.default_rng(4)
    q, K, V = rng.normal(size=(2, 64)), rng.normal(size=(9, 64)), rng.normal(size=(9, 64))
    O, lse, P = oracle.decode_attention(q, K, V)
    O2, lse2 = oracle.attention_rows(q, K, V, oracle.scale_for(64))
    np.testing.assert_allclose(O, O2, rtol=1e-13)
    np.testing.assert_allclose(lse, lse2, rtol=1e-13)
    np.testing.assert_allclose(P.sum(axis=1), 1.0, rtol=1e-14)
    O, lse, P = oracle.decode_attention(q, K[:0], V[:0])
    assert (O == 0).all() and np.isneginf(lse).all() and P.shape == (2, 0)


@pytest.mark.parametrize("budget,n_first,n_recent,holes,fills", [
    (3, 0, 0, [0, 2], [3, 5]),     # masses 9, 8, 7 at 3, 1, 5
    (3, 1, 0, [2], [3]),           # token 0 held: 0, 3, 1
    (3, 1, 2, [1, 2], [4, 5]),     # 0, 4, 5 held
    (1, 0, 0, [0], [3]),
    (6, 0, 0, [], []),
])
def test_evict_plan_by_hand(budget, n_first, n_recent, holes, fills):
    mass = [1, 8, 2, 9, 0, 7]
    assert oracle.evict_plan(mass, None, budget, n_first, n_recent) == (holes, fills)


def test_evict_plan_ties_nan_and_moved_positions():
    assert oracle.evict_plan([5, 5, 5, 5], None, 2, 0, 0) == ([], [])      # ties: lower index
    assert oracle.evict_plan([np.nan, 1, 1, 2], None, 2, 0, 0) == ([0], [3])
    assert oracle.evict_plan([-np.inf, np.nan, 0, -1], None, 3, 0, 0) == ([1], [3])
    # the newest token (largest position) sits at index 0
    assert oracle.evict_plan([0, 3, 2, 1], [9, 0, 1, 2], 2, 0, 1) == ([], [])
    assert oracle.evict_plan([0, 1, 2, 3], [9, 0, 1, 2], 2, 0, 1) == ([1], [3])


def test_compact_rows_moves_through_the_page_table():
    pool = np.arange(3 * 1 * 4 * 1, dtype=float).reshape(3, 1, 4, 1)
    ref = pool.copy()
    oracle.compact_rows(pool, [2, 0], 0, [1], [5], 4)   # row 5 = slot 0 row 1 -> slot 2 row 1
    assert pool[2, 0, 1, 0] == ref[0, 0, 1, 0]
    pool[2, 0, 1] = ref[2, 0, 1]
    assert np.array_equal(pool, ref)
