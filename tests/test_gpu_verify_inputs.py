"""Verification of drafted trees on rows of any content against verify_ref.py: what a draft's buffer holds where nobody drew
from it, NaN, negative and infinite draft probabilities, greedy rows without probability."""
import math

import pytest
import torch

import semantic_paged_kv_gb300 as ice
import verify_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _rows(B, T, V, dtype, seed):
    z = 2 * torch.randn((B, T, V), generator=_gen(seed), device="cuda")
    w = z + torch.randn((B, T, V), generator=_gen(seed + 1), device="cuda")
    return torch.softmax(z, -1).to(DT[dtype]), torch.softmax(w, -1).to(DT[dtype])


def _tree(B, T, wide, seed):
    g = torch.Generator().manual_seed(seed)
    p = [[-1] + [int(torch.randint(0, min(t, wide), (1,), generator=g)) for t in range(1, T)] for _ in range(B)]
    return torch.tensor(p, dtype=torch.int32, device="cuda")


def _drawn(draft, parents, seed):
    """A token for every node, from its parent's row."""
    q = draft.float().gather(1, parents.clamp(min=0).long()[..., None].expand(*parents.shape, draft.shape[-1]))
    return (q / torch.empty_like(q).exponential_(generator=_gen(seed))).argmax(-1).int()


def _run(target, draft, tokens, parents, counts, uniform):
    B, T = tokens.shape
    path = torch.full((B, T), 99, dtype=torch.int32, device="cuda")
    n, nxt, err = (torch.full((k,), x, dtype=torch.int32, device="cuda") for k, x in ((B, 99), (B, 99), (1, 0)))
    ice.ice_tree_verify(ice.Tree(parents, counts, T), ice.probs(target), None if draft is None else ice.probs(draft),
                        tokens, uniform, path, n, nxt, err)
    return path, n, nxt, ice.ice_check(err)


def _check(target, draft, tokens, parents, counts, uniform, status=ice.ICE_OK):
    path, n, nxt, got = _run(target, draft, tokens, parents, counts, uniform)
    assert got == status
    B, T = tokens.shape
    near_border = 0
    for b in range(B):
        m = T if counts is None else int(counts[b])
        want, x, near = verify_ref.verify(target[b].double().cpu(), None if draft is None else draft[b].double().cpu(),
                                          tokens[b].tolist(), None if parents is None else parents[b].tolist(),
                                          None if uniform is None else uniform[b].double().tolist(), m)
        if near < 1e-11:  # sums in another order may decide otherwise
            near_border += 1
            continue
        assert path[b].tolist() == want + [-1] * (T - len(want)), b
        assert int(n[b]) == len(want) and int(nxt[b]) == x, b
    assert near_border == 0


def test_a_root_alone_takes_the_target_whatever_the_draft_holds():
    p = torch.tensor([[[0.7, 0.2, 0.1]]], device="cuda")
    zero = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for bad in (math.nan, math.inf, -math.inf, -3.0, 1e38):
        q = torch.tensor([[[bad, 0.5, 0.5]]], device="cuda")
        for u, want in ((0.1, 0), (0.75, 1), (0.95, 2)):
            path, n, nxt, err = _run(p, q, zero, None, None, torch.full((1, 1), u, device="cuda"))
            assert err == ice.ICE_OK and path.tolist() == [[0]] and int(n) == 1 and int(nxt) == want


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("B,T,V,wide", [(24, 17, 40, 17), (16, 40, 333, 3), (4, 26, 4099, 2), (2, 61, 32003, 4)])
def test_draft_of_any_content(B, T, V, wide, offset, dtype):
    """NaN, negative and infinite numbers all over the draft (and NaN and negative ones in the target), at drafted tokens too;
    rows of the draft that start elsewhere in a vector than the target's."""
    target, clean = _rows(B, T, V, dtype, 7)
    parents = _tree(B, T, wide, 8)
    tokens = _drawn(clean, parents, 9)
    uniform = torch.rand((B, T), generator=_gen(10), device="cuda").clamp(min=2.0 ** -24)
    counts = torch.tensor([T - (b * 5) % T for b in range(B)], dtype=torch.int32, device="cuda")
    big = torch.zeros((B, T, V + offset), dtype=DT[dtype], device="cuda")
    draft = big[..., offset:]
    draft.copy_(clean)
    _check(target, draft, tokens, parents, counts, uniform)  # as it should be
    what = torch.rand((B, T, V), generator=_gen(11), device="cuda")
    for lo, x in ((0.0, math.nan), (0.05, -0.4), (0.1, math.inf), (0.12, -math.inf)):
        draft.masked_fill_((what >= lo) & (what < lo + 0.05), x)
    # at drafted tokens more often: every other node's
    at = torch.arange(B * T, device="cuda").view(B, T) % 4
    for k, x in ((0, math.nan), (1, -0.3)):
        b, t = ((at == k) & (parents >= 0)).nonzero(as_tuple=True)
        draft[b, parents[b, t].long(), tokens[b, t].long()] = x
    _check(target, draft, tokens, parents, counts, uniform)
    what = torch.rand((B, T, V), generator=_gen(12), device="cuda")
    target.masked_fill_(what < 0.05, math.nan).masked_fill_(what > 0.95, -0.7)
    _check(target, draft, tokens, parents, counts, uniform)
    _check(target, None, tokens, parents, counts, uniform)
    _check(target, None, tokens, parents, counts, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_nobody_drew_from_are_not_read(dtype):
    """The draft's rows of nodes without children hold NaN throughout, or infinities: the same answers."""
    B, T, V = 40, 9, 5000
    target, draft = _rows(B, T, V, dtype, 17)
    parents = _tree(B, T, 3, 18)
    tokens = _drawn(draft, parents, 19)
    uniform = torch.rand((B, T), generator=_gen(20), device="cuda")
    want = _run(target, draft, tokens, parents, None, uniform)
    leaf = torch.ones((B, T), dtype=torch.bool, device="cuda")
    leaf.scatter_(1, parents.clamp(min=0).long(), False)
    reached = want[0].gather(1, (want[1] - 1)[:, None].long())
    assert int(leaf.gather(1, reached.long()).sum()) > 5  # walks that end there
    for x in (math.nan, math.inf, -1.0):
        got = _run(target, draft.masked_fill(leaf[..., None], x), tokens, parents, None, uniform)
        assert got[3] == ice.ICE_OK and all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    # all but one element of a leaf's row: none of the target's is lost
    some = draft.masked_fill(leaf[..., None], math.nan)
    some[..., 4321] = torch.where(leaf, torch.full_like(some[..., 0], 0.5), some[..., 4321])
    got = _run(target, some, tokens, parents, None, uniform)
    assert got[3] == ice.ICE_OK and all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 50, 5003])
def test_greedy_rows_without_probability(V, dtype):
    """Zeros, negative numbers and NaN alone: no child is accepted there, -1 follows, and the call says so."""
    B, T = 6, 4
    target, _ = _rows(B, T, V, dtype, 27)
    parents = torch.tensor([[-1, 0, 1, 2]] * B, dtype=torch.int32, device="cuda")
    best = target.argmax(-1).int()
    tokens = torch.cat((best[:, :1], best[:, :-1]), 1).contiguous()  # every drafted token is the likeliest
    target[1, 0], target[2, 1], target[3, 3], target[4, 2] = 0, -0.25, math.nan, 0
    target[4, 2, ::2] = math.nan
    for b, i in ((1, 1), (2, 2), (4, 3)):
        tokens[b, i] = 0  # the first of the largest, if 0 counted
    path, n, nxt, err = _run(target, None, tokens, parents, None, None)
    assert err == ice.ICE_ERR_INVALID_ARG
    assert n.tolist() == [4, 1, 2, 4, 3, 4] and [nxt[b].item() for b in (1, 2, 3, 4)] == [-1] * 4
    assert nxt[0] == best[0, 3] and nxt[5] == best[5, 3]
    keep = torch.tensor([0, 5], device="cuda")
    _check(target[keep], None, tokens[keep], parents[keep], None, None)
    _check(target, None, tokens, parents, None, None, ice.ICE_ERR_INVALID_ARG)
