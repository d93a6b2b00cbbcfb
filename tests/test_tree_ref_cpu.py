"""The restatement of the verification against direct enumeration, and mistakes planted in it."""
import pytest
import torch

import tree_ref as ref


def _step(p, q, tokens, u):
    """One node and its children by renormalising after every refusal."""
    r = p.clone()
    for c, x in enumerate(tokens[1:], 1):
        if u[c] * float(q[x]) < float(r[x]):
            return [0, c]
        r = (r - q).clamp(min=0)
        r = r / r.sum()
    return [0]


@pytest.mark.parametrize("seed", range(20))
def test_one_node_as_renormalised(seed):
    g = torch.Generator().manual_seed(seed)
    V, T = 9, 6
    p, q = (torch.softmax(2 * torch.randn(T, V, generator=g, dtype=torch.float64), -1) for _ in range(2))
    tokens = torch.multinomial(q[0], T, replacement=True, generator=g).tolist()
    u = torch.rand(T, generator=g, dtype=torch.float64).tolist()
    path, nxt, near = ref.verify(p, q, tokens, [-1] + [0] * (T - 1), u, T)
    assert near > 1e-12 and path == _step(p[0], q[0], tokens, u) and 0 <= nxt < V


def test_the_target_distribution_is_kept():
    """The probability of every first token, by integrating over drafted tokens and accept decisions on a grid of
    random numbers, is the target's; without the residual (drawing from p again) it is not."""
    V, N = 4, 400
    p = torch.tensor([[0.4, 0.3, 0.2, 0.1]] * 2, dtype=torch.float64)
    q = torch.tensor([[0.1, 0.2, 0.3, 0.4]] * 2, dtype=torch.float64)
    got, naive = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
    for x in range(V):
        accept = min(1.0, float(p[0, x] / q[0, x]))
        for i in range(N):
            u = (i + 0.5) / N
            path, nxt, _ = ref.verify(p, q, [0, x], [-1, 0], [0.0, u], 2)
            assert (len(path) == 2) == (u < accept)
            w = float(q[0, x]) / N
            if len(path) == 2:
                got[x] += w
                naive[x] += w
            else:
                for j in range(50):
                    got[ref.verify(p, q, [0, x], [-1, 0], [(j + 0.5) / 50, u], 2)[1]] += w / 50
                naive += w * p[0]
    assert float((got - p[0]).abs().max()) < 0.01
    assert float((naive - p[0]).abs().max()) > 0.05


def test_sees():
    m = ref.sees([-1, 0, 0, 1, -1], 5)
    assert m.int().tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    assert torch.equal(ref.sees(None, 4), torch.ones(4, 4, dtype=torch.bool).tril())


def test_masked_values_take_no_part():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(3, 128, generator=g, dtype=torch.float64) for _ in range(3))
    keep = ref.sees(None, 3)
    want = ref.attention(q, k, v, keep, 0.1)
    v2 = v.clone()
    v2[2] = float("inf")
    got = ref.attention(q, k, v2, keep, 0.1)
    assert torch.allclose(got[:2], want[:2], rtol=1e-13, atol=0) and bool(torch.isinf(got[2]).all())


def test_tolerance_notices_a_missing_token():
    """A node that does not see one of its ancestors, or sees another branch, is out of bounds."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(12, 128, generator=g, dtype=torch.float64) for _ in range(3))
    keep = ref.sees([-1, 0, 0, 1, 1, 2, 3, 3, 4, 5, 6, 9], 12)
    want, tol = ref.attention(q, k, v, keep, 0.088), ref.tolerance(q, k, v, keep, 0.088, torch.bfloat16)
    wrong = keep.clone()
    wrong[6, 1] = False
    wrong[8, 2] = True
    off = (ref.attention(q, k, v, wrong, 0.088) - want).norm(dim=-1)
    assert bool((off[[6, 8]] > tol[[6, 8]]).all()) and float(off[[0, 3, 11]].max()) == 0
