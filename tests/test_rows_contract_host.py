"""Promises of the header on draft verification that the oracle has to keep too (no GPU)."""

import numpy as np
import pytest

from oracle import kvq_paged_oracle as P

NAN, INF = float("nan"), float("inf")
# p and q of the drafted token, u, and whether the draft stands: u q < p, where a
# probability that is not above 0 (NaN too) counts as 0 and one above 1 as 1
ODD = [
    (0.0, -0.5, 0.5, False),         # 0 < 0
    (0.0, -INF, 0.5, False),
    (0.0, NAN, 0.5, False),
    (-1.0, -2.0, 0.75, False),
    (-1.0, 0.5, 0.0, False),
    (NAN, 0.5, 0.0, False),
    (NAN, NAN, 0.0, False),
    (0.25, NAN, 0.5, True),          # 0 < 1/4
    (0.25, -1.0, 0.999, True),
    (0.25, INF, 0.0, True),          # u < 1/4
    (0.25, INF, 0.125, True),
    (0.25, 2.0, 0.1875, True),
    (0.25, 2.0, 0.25, False),
    (0.25, INF, 0.5, False),
    (2.0, 1.0, 0.999, True),         # u < 1
    (INF, INF, 0.999, True),
    (INF, 0.5, 0.999, True),
    (0.5, 0.5, 0.999, True),         # as ever
    (0.25, 0.5, 0.5, False),
]


def odd_rows(p, q, u):
    """One sequence with one draft, token 2: where it falls the next token is 4, where it stands 6."""
    target, draft = np.zeros((2, 8)), np.zeros((1, 8))
    target[0, 2], draft[0, 2], target[0, 4], target[1, 6] = p, q, 0.5, 1.0
    return target, draft, np.array([2], np.int32), np.array([u, 0.9999])


@pytest.mark.parametrize("p,q,u,stands", ODD)
def test_probabilities_of_a_draft_that_are_none(p, q, u, stands):
    assert P.verify(*odd_rows(p, q, u)) == ((2, 6) if stands else (1, 4))
