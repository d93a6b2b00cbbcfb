"""The restatement for rows of any content against examples by hand."""
import math

import pytest
import torch

import tree_ref
import verify_ref

F = torch.float64


def test_draft_values_that_count_as_nothing():
    p = torch.tensor([[0.7, 0.2, 0.1]] * 2, dtype=F)
    for bad in (math.nan, -0.5, -math.inf):
        q = torch.tensor([[bad, 0.5, 0.5]] * 2, dtype=F)
        # no child: the target's own distribution
        assert verify_ref.verify(p, q, [0], None, [0.1], 1)[:2] == ([0], 0)
        # token 0 with q = 0 is accepted whatever its random number
        assert verify_ref.verify(p, q, [0, 0], None, [0.1, 0.999], 2)[0] == [0, 1]
        # token 1 is refused (0.9 of 0.5 against 0.2); what is left is max(p - q, 0) = (0.7, 0, 0)
        assert verify_ref.verify(p, q, [0, 1], None, [0.999, 0.9], 2)[:2] == ([0], 0)
        # a token of no probability is not accepted for a negative q
        z = torch.tensor([[0.0, 0.9, 0.1]] * 2, dtype=F)
        assert verify_ref.verify(z, q, [0, 0], None, [0.5, 0.5], 2)[:2] == ([0], 1)
    q = torch.tensor([[math.inf, 0.1, 0.1]] * 2, dtype=F)
    assert verify_ref.verify(p, q, [0], None, [0.1], 1)[:2] == ([0], 0)
    assert verify_ref.verify(p, q, [0, 0], None, [0.1, 0.5], 2)[:2] == ([0], 1)  # refused, nothing left of it


def test_greedy_rows_without_probability():
    for row in ([0.0, 0.0], [-1.0, 0.0], [math.nan, -2.0], [math.nan, math.nan]):
        p = torch.tensor([row] * 2, dtype=F)
        assert verify_ref.verify(p, None, [0, 0], None, None, 2)[:2] == ([0], -1)
    p = torch.tensor([[math.nan, 0.1, -3.0, 0.1]] * 2, dtype=F)
    assert verify_ref.verify(p, None, [0, 1], None, None, 2)[:2] == ([0, 1], 1)


@pytest.mark.parametrize("seed", range(10))
def test_rows_of_probabilities_as_before(seed):
    g = torch.Generator().manual_seed(seed)
    V, T = 9, 6
    p, q = (torch.softmax(2 * torch.randn(T, V, generator=g, dtype=F), -1) for _ in range(2))
    tokens = torch.multinomial(q[0], T, replacement=True, generator=g).tolist()
    u = torch.rand(T, generator=g, dtype=F).tolist()
    for draft, uniform in ((q, u), (None, u), (None, None)):
        assert verify_ref.verify(p, draft, tokens, [-1] + [0] * (T - 1), uniform, T) == \
            tree_ref.verify(p, draft, tokens, [-1] + [0] * (T - 1), uniform, T)
