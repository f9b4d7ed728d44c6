"""Pins of the serving oracle: closed forms, enumeration and invariants."""
import numpy as np
import pytest

from oracle import dustin_oracle as O
from oracle import serving_oracle as S


def test_accepting_and_drawing_reproduce_the_target_distribution():
    """Over a fine grid of (u_accept, u_sample) and drafts drawn from q, the
    first token's frequencies are the target's probabilities."""
    p = np.array([0.5, 0.125, 0.25, 0.125])
    q = np.array([0.25, 0.5, 0.125, 0.125])
    grid = (np.arange(64) + 0.5) / 64
    got = np.zeros(4)
    for x in range(4):
        for ua in grid:
            for us in grid:
                t, _ = S.verify_tokens(np.array([[p, p]]), np.array([[q]]), np.array([[x]]), None,
                                       np.array([[ua]]), np.array([us]))
                got[t[0, 0]] += q[x] / 64 ** 2
    np.testing.assert_allclose(got, p, atol=1 / 64)


def test_all_drafts_accepted_draws_from_the_last_row():
    p = np.zeros((1, 3, 5))
    p[0, 0, 2] = p[0, 1, 3] = p[0, 2, 4] = 1.0
    t, a = S.verify_tokens(p, p[:, :2], np.array([[2, 3]]), None, np.array([[0.9, 0.9]]),
                           np.array([0.3]))
    assert t.tolist() == [[2, 3, 4]] and a.tolist() == [2]


def test_certain_drafts_and_empty_residuals():
    p = np.array([[[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]])
    t, a = S.verify_tokens(p, None, np.array([[0]]), None, np.array([[0.6]]), np.array([0.0]))
    assert t.tolist() == [[1, -1]] and a.tolist() == [0]        # 0 is rejected, so drawn from {1}
    t, a = S.verify_tokens(p, p[:, :1], np.array([[0]]), None, np.array([[1.0]]), np.array([0.9]))
    assert t.tolist() == [[1, -1]]                              # p - q is empty: p itself
    t, a = S.verify_tokens(0 * p, None, np.array([[0]]), None, np.array([[0.0]]), np.array([0.9]))
    assert t.tolist() == [[-1, -1]]


@pytest.mark.parametrize("u,want", [(0.0, 1), (0.249, 1), (0.25, 3), (0.999, 3), (1.0, 3),
                                    (float("nan"), 1)])
def test_draw_by_inversion(u, want):
    assert S.draw(np.array([0.0, 0.25, 0.0, 0.75, 0.0]), u) == want


def test_pages_are_shared_copied_and_returned():
    book = S.PageBook([[5, 2, -1, -1]] + [[-1] * 4] * 3, [20, 0, 0, 0],
                      [0, 0, 1, 0, 0, 1, 0, 0], 16)
    assert book.consistent()
    assert book.fork([0, 0, 0], [1, 2, 1]) == [2]               # child 1 named twice
    assert book.consistent() and book.table[2][:2] == [5, 2] and book.refcount[2] == 3
    copies, starved = book.resize([1, 2], [40, 21])
    assert copies == [[2, 0], [2, 3]] and starved == []
    assert book.consistent() and book.table[1] == [5, 0, 1, -1]
    copies, starved = book.resize([1, 2, 0], [0, 17, 64])
    assert copies == [[-1, -1]] * 3 and starved == []           # 0's page is its own again
    assert book.consistent() and book.table[0] == [5, 2, 0, 1]
    # 0 gives back three pages first; six are free: enough for 3, not for 1.
    assert book.resize([3, 1, 0], [64, 64, 5])[1] == [1] and book.consistent()
    assert book.seq_len == [5, 0, 17, 64] and book.table[3] == [0, 1, 2, 4]


def test_compaction_of_everything_is_the_identity():
    x = np.arange(2 * 3 * 7 * 2.0).reshape(2, 3, 7, 2)
    idx = np.tile(np.arange(7), (2, 1))
    assert np.array_equal(S.compact(x, idx, None, x.copy()), x)
    got = S.compact(x, idx[:, 3:5], [2, 1], np.zeros((2, 3, 2, 2)))
    assert np.array_equal(got[0], x[0, :, 3:5]) and not got[1, :, 1].any()


def test_prefix_attention_is_full_attention_over_joined_keys():
    r = np.random.default_rng(0)
    q = r.standard_normal((4, 4, 3, 8))
    kp, vp = r.standard_normal((2, 2, 11, 8)), r.standard_normal((2, 2, 11, 8))
    ko, vo = r.standard_normal((4, 2, 5, 8)), r.standard_normal((4, 2, 5, 8))
    o, lse = S.prefix_attention(q, kp, vp, ko, vo, 2, 0.3)
    k = np.concatenate([np.repeat(kp, 2, 0), ko], 2)
    v = np.concatenate([np.repeat(vp, 2, 0), vo], 2)
    ro, rl = O.full_verify_attention(q, k, v, 0.3)
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    o, lse = S.prefix_attention(q, kp, vp, ko, vo, 2, 0.3, prefix_len=[0, 0], own_len=[0] * 4)
    assert not o.any() and np.all(np.isneginf(lse))


@pytest.mark.parametrize("p,q,want", [(-0.25, -0.75, 0), (float("inf"), 0.5, 0), (float("nan"), 0.0, 0),
                                      (0.0, -1.0, 0), (0.5, float("nan"), 1), (0.5, float("inf"), 1)])
def test_entries_without_mass_count_as_zero_in_the_acceptance(p, q, want):
    rows = np.array([[[p, 0.5], [0.0, 1.0]]])
    _, a = S.verify_tokens(rows, np.array([[[q, 0.5]]]), np.array([[0]]), None, np.array([[0.9]]),
                           np.array([0.0]))
    assert a.tolist() == [want]
