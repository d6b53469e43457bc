"""The oracle of pages, rotary positions and prompt attention, held against
hand-derived cases and against properties that it does not compute by."""
import numpy as np
import pytest

from oracle import kv_oracle as KO
from oracle import prompt_oracle as PO


def test_pages_are_taken_in_order_and_put_back_the_other_way_round():
    free, table, held = [9, 8, 7, 6, 5] + 5 * [0], [[0, 0, 0], [1, 2, 0]], [0, 2]
    # 33 tokens need 3 pages of 16, 17 need 2: the stack's top goes first
    count, slots, positions, flags = PO.assign(free, 5, table, held, [0, 16], 16, [33, 1], [0, 33], 34, 40)
    assert count == 2 and held == [3, 2] and table == [[5, 6, 7], [1, 2, 0]] and flags == [0, 0]
    assert slots[0] == 5 * 16 and slots[32] == 7 * 16 and slots[33] == 2 * 16 and positions[33] == 16
    count, _, _, _ = PO.assign(free, count, table, held, [0, 32], 16, [0, 0], [0, 0], 0, 0)
    assert count == 5 and free[:5] == [9, 8, 7, 6, 5] and held == [0, 2]


def test_a_sequence_that_lacks_too_many_stops_the_later_ones():
    free, table, held = [4, 3, 2] + 5 * [0], [[0] * 4, [0] * 4, [7, 0, 0, 0]], [0, 0, 1]
    count, slots, _, flags = PO.assign(free, 3, table, held, [0, 0, 0], 16, [16, 64, 16], [0, 16, 80], 96, 64)
    assert flags == [0, PO.NO_PAGE, 0] and held == [1, 0, 1] and count == 2
    assert slots[16] == -1 and slots[80] == 7 * 16
    held, table = [0, 0, 0], [[0] * 4 for _ in range(3)]
    count, slots, _, flags = PO.assign([4, 3, 2] + 5 * [0], 3, table, held, [0, 0, 0], 16, [16, 64, 16], [0, 16, 80], 96, 64)
    assert flags == [0, PO.NO_PAGE, PO.NO_PAGE] and held == [1, 0, 0]


def test_no_page_is_lost_or_given_twice():
    g = np.random.default_rng(0)
    size, batch, page, columns = 60, 7, 16, 20
    free, table, held, count = list(range(size)), [[0] * columns for _ in range(batch)], [0] * batch, size
    for _ in range(200):
        ctx, new = g.integers(0, 200, batch).tolist(), g.integers(0, 100, batch).tolist()
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        count, _, _, _ = PO.assign(free, count, table, held, ctx, page, new, starts, starts[-1], 100)
        owned = [table[b][c] for b in range(batch) for c in range(held[b])]
        assert sorted(owned + free[:count]) == list(range(size))


def test_positions_of_a_tree():
    parents = [-1, 0, 0, 1, 3, 2]
    _, _, positions, flags = PO.assign([3, 2, 1, 0], 4, [[0, 0]], [0], [10], 16, [6], [0], 6, 6, parents)
    assert [positions[i] - 10 for i in range(6)] == [0, 1, 1, 2, 3, 2] and flags == [0]


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_scores_depend_on_the_distance_alone(adjacent):
    g = np.random.default_rng(1)
    freq = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    q, k = g.normal(size=(1, 1, 20)), g.normal(size=(1, 1, 20))
    score = lambda i, j: float((PO.rope(q, [[i]], freq, [0] * 8, adjacent)[0] * PO.rope(k, [[j]], freq, [0] * 8, adjacent)[0]).sum())
    assert abs(score(5, 3) - score(1005, 1003)) < 1e-9 and abs(score(5, 3) - score(6, 3)) > 1e-3
    turned, size = PO.rope(q, [[77]], freq, [0] * 8, adjacent)
    np.testing.assert_allclose(np.linalg.norm(turned), np.linalg.norm(q), rtol=1e-12)
    assert (turned[..., 16:] == q[..., 16:]).all() and (size[..., 16:] == 0).all()


def test_rotary_pairs_and_axes_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    c, s = np.cos(2.0), np.sin(2.0)
    # pair 0 turns with the second axis (position 2), pair 1 with the first (position 0)
    got, _ = PO.rope(x, [[0], [2]], [1.0, 1.0], [1, 0], False)
    np.testing.assert_allclose(got[0, 0], [c - 3 * s, 2, s + 3 * c, 4], atol=1e-15)
    got, _ = PO.rope(x, [[0], [2]], [1.0, 1.0], [1, 0], True)
    np.testing.assert_allclose(got[0, 0], [c - 2 * s, s + 2 * c, 3, 4], atol=1e-15)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 0), (5, 3), (2, 40), (100, 1)])
def test_a_prompt_sees_what_a_chain_over_an_empty_cache_sees(window, sinks):
    assert (PO.sees(17, window, sinks) == KO.visible(0, 17, None, window, sinks)).all()


def test_attention_by_hand():
    q, k, v = np.zeros((3, 2, 4)), np.ones((3, 1, 4)), np.arange(3.0)[:, None, None] * np.ones((3, 1, 4))
    out, lse, absolute, _ = PO.attention(q, k, v, 0.5, 0, 0)  # even weights
    np.testing.assert_allclose(out[:, 0, 0], [0, 0.5, 1.0])
    np.testing.assert_allclose(lse[:, 1], np.log([1, 2, 3]))
    q[2] = 1000.0
    k[1] = 2.0
    out, _, _, _ = PO.attention(q, k, v, 0.5, 0, 0)  # all weight on token 1
    np.testing.assert_allclose(out[2], 1.0)
    v[2], k[2] = np.nan, np.inf
    out, lse, _, _ = PO.attention(q, k, v, 0.5, 0, 0)
    assert np.isfinite(out[:2]).all() and np.isfinite(lse[:2]).all()
