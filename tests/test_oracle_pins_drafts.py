"""Pins of the drafts' oracle: entries of the draft rows that are no probabilities."""
import numpy as np

from oracle import hybrid as ho

NAN = float("nan")


def _draw(target, draft, u):
    """The next token after a draft of token 0 that u_accept = 1 rejects (target 0 < draft 1 there)."""
    p, q = np.array([target, [0.0] * len(target)]), np.array([draft])
    a, nxt = ho.accept_drafts(p, [[0]], np.array([[1.0]]), [u], q)
    assert a[0] == 0
    return nxt[0]


def test_a_nan_draft_entry_counts_as_nothing():
    # r = (0, .25, .25): the NaN takes nothing from token 1
    assert [_draw([0.0, 0.25, 0.25], [1.0, NAN, 0.0], u) for u in (0.0, 0.49, 0.5, 0.99)] == [1, 1, 2, 2]


def test_a_negative_draft_entry_adds_nothing():
    # r = (0, .25, .25), not (0, 1, .25)
    assert [_draw([0.0, 0.25, 0.25], [1.0, -0.75, 0.0], u) for u in (0.0, 0.49, 0.5, 0.99)] == [1, 1, 2, 2]


def test_a_token_without_target_probability_is_never_drawn():
    # r = (0, 0, 0, .25): neither a zero nor a negative target entry gains from a more negative draft entry
    assert [_draw([0.0, 0.0, -0.25, 0.25], [1.0, -0.5, -0.75, 0.0], u) for u in (0.0, 0.5, 0.99)] == [3, 3, 3]


def test_without_a_positive_residual_the_target_row_is_drawn_from():
    # p - q is positive for token 1 only through its negative draft entry
    assert [_draw([0.0, 0.0, 0.5, 0.5], [1.0, -0.5, 0.5, 0.75], u) for u in (0.0, 0.49, 0.5, 0.99)] == [2, 2, 3, 3]
