"""Pins of oracle/draft.py: hand cases, the fallbacks, and that the rule leaves
the target's distribution unchanged (by integration over a grid of u)."""

import numpy as np

from oracle import draft


def test_hand_case():
    p = np.array([[0.5, 0.25, 0.25], [0.125, 0.125, 0.75], [0.25, 0.5, 0.25]])
    q = np.array([[0.25, 0.5, 0.25], [0.75, 0.125, 0.125]])
    # token 0 stays (0.9 * 0.25 < 0.5); token 0 of the second row: 0.5 * 0.75 >= 0.125, refused;
    # rest = (0, 0, 0.625): the next token is 2
    assert draft.verify(p, q, [0, 0], 2, [0.9, 0.5], 0.99) == ([0, 2, -1], 1)
    # all stay: drawn from the extra row, 0.25 < 0.3 * 1 -> entry 1
    assert draft.verify(p, q, [0, 2], 2, [0.9, 0.9], 0.3) == ([0, 2, 1], 2)
    # a shorter draft: the row after it is the extra one
    assert draft.verify(p, q, [0, 0], 1, [0.9, 0.5], 0.1) == ([0, 0, -1], 1)
    # the border itself is refused (u q < p is strict), and passes a running sum (strict)
    assert draft.verify(p, q, [1, 0], 2, [0.5, 0.0], 0.0)[1] == 0
    assert draft.verify(p, None, [1, 0], 0, [0.5, 0.0], 0.5) == ([1, -1, -1], 0)


def test_greedy_draft_leaves_the_token_out():
    p = np.array([[0.5, 0.25, 0.25], [1.0, 0.0, 0.0]])
    assert draft.verify(p, None, [0], 1, [0.5], 0.0) == ([1, -1], 0)
    assert draft.verify(p, None, [0], 1, [0.49], 0.9) == ([0, 0], 1)


def test_fallbacks():
    p = np.array([[0.0, 1.0, 0.0], [0.0, 0.0, 0.0]])
    q = np.array([[0.0, 1.0, 0.0]])
    # token 2 has p = 0: refused, nothing is left of p - q, so p itself
    assert draft.verify(p, q, [2], 1, [0.5], 0.5) == ([1, -1], 0)
    assert draft.verify(p, q, [1], 1, [0.5], 0.5) == ([1, 2], 1)      # an empty row: its last entry
    assert draft.verify(p, q, [-1], 1, [0.0], 0.5) == ([1, -1], 0)    # not a token
    assert draft.verify(p, q, [3], 1, [0.0], 0.5) == ([1, -1], 0)
    bad = np.array([[np.nan, np.inf, 0.25], [0.5, 0.5, 0.0]])
    assert draft.verify(bad, None, [0], 1, [0.0], 0.9) == ([2, -1], 0)


def test_target_distribution_is_kept():
    p = np.array([[0.5, 0.375, 0.125], [1.0, 0.0, 0.0]])
    q = np.array([[0.25, 0.5, 0.25]])
    n = 64
    count = np.zeros(3)
    for x in range(3):
        for i in range(n):
            for j in range(n):
                t, _ = draft.verify(p, q, [x], 1, [(i + 0.5) / n], (j + 0.5) / n)
                count[t[0]] += q[0, x] / n / n
    assert np.allclose(count, p[0], atol=1.5 / n)
