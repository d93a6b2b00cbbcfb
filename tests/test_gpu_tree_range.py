"""Attention of drafted trees at the ends of the number ranges: scores whose keys, queries or scale are near fp32's ends, values
near the largest that a sum holds, infinities and NaN of nodes that weigh nothing, elements far below their row's largest."""
import math

import pytest
import torch

import cache4_ref as ref4
import semantic_paged_kv_gb300 as ice
import tree_ref as ref
from test_gpu_tree import D, S, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ks,qs,scale", [
    (1e34, 1e-34, None), (1e35, 1e-35, None), (3e36, 1e-37, None), (1e-36, 1e36, None), (1e-30, 1e35, 1e-6),
    (1e36, 1.0, 1e-37), (1.0, 1e36, 1e-37), (1e18, 1e18, 1e-37), (1e-18, 1e-18, 1e35), (1e33, 1e-36, 1e2)])
def test_scores_at_the_ends_of_the_range(ks, qs, scale, dtype):
    """Keys, queries and scale far apart whose scores are ordinary: rows of cached tokens, of nodes, and of runs that are joined."""
    for lens in ([200, 33], [5000, 0]):
        c = Case(2, 9, 8, 2, dtype, True, lens, seed=7, k_scale=ks, q_scale=qs)
        if scale:
            c.scale = scale
        c.run()
        assert ice.ice_check(c.err) == ice.ICE_OK
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_keys_of_very_different_size(dtype):
    """A few keys beyond 2^112 among ordinary ones that are tiny beside them, with queries that make the large ones ordinary."""
    c = Case(2, 9, 8, 2, dtype, True, [300, 40], seed=11, q_scale=1e-34)
    big = torch.tensor([1e34 if i % 5 == 0 else 1.0 for i in range(c.recs.shape[0])], device="cuda")
    k, v = ref4.decode(c.recs.view(-1, 2304))
    fine = torch.isfinite(k).all(-1).all(-1) & torch.isfinite(v).all(-1).all(-1)
    k = (torch.nan_to_num(k).view(-1, c.hkv, S, D) * big[:, None, None, None]).view(-1, S, D)
    new = ref4.encode(k.bfloat16(), torch.nan_to_num(v).bfloat16())
    c.recs.copy_(torch.where(fine[:, None], new, c.recs.view(-1, 2304)).view_as(c.recs))
    c.k[:, ::3] *= 1e34
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_values_of_long_sequences(dtype):
    """The largest |v| times the number of tokens just below 2^119, in segments that runs cut, with scores that rise by 7.9
    powers of two inside the first run alone: its weights are the largest, and all of them count."""
    B, hkv, n = 25, 4, 8192
    c = Case(B, 1, hkv, hkv, dtype, False, [n] * B, counts=[1] * B)
    x = torch.zeros((2, S, D), device="cuda")
    x[1, :, 0] = 1.0  # scores of 0 and, below, of 7.9 log 2
    sign = torch.where(torch.arange(D, device="cuda") % 3 == 0, -1.0, 1.0)
    v = (2.0 ** 105 * sign).expand(2, S, D).clone()
    v[..., 64:] = 2.0 ** 105  # (groups of one value are exact in 4 bits; the first one holds two)
    low, high = ref4.encode(x.bfloat16(), v.bfloat16())
    c.recs[:] = low
    for b in range(B):
        c.recs[c.table[b, 8:168].long()] = high  # tiles 1 .. 20 of the 64
    c.q.zero_()
    c.q[..., 0] = 62.0
    c.k.zero_()
    c.v.copy_((2.0 ** 105 * sign).expand_as(c.v))
    c.v[..., 64:] = 2.0 ** 105
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK and bool(torch.isfinite(c.O).all())
    k0, v0 = c.cached(0, 0)
    k1, v1 = torch.cat((k0, c.k[0, :, 0].double())), torch.cat((v0, c.v[0, :, 0].double()))
    keep = torch.ones((1, n + 1), dtype=torch.bool, device="cuda")
    q = c.q[0, :, 0].double()
    want, tol = ref.attention(q, k1, v1, keep, c.scale), ref.tolerance(q, k1, v1, keep, c.scale, c.dt)
    off = (c.O.double() - want).norm(dim=-1)  # (all units have the same inputs)
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,hq,hkv,lens", [(1, 8, 2, [5000]), (1, 8, 2, [20000]), (2, 8, 2, [100, 0]), (60, 8, 2, [40] * 60),
                                           (3, 32, 8, [900, 0, 300]), (100, 4, 1, [8192] * 100)])
def test_infinities_of_nodes_that_weigh_nothing(B, hq, hkv, lens, dtype):
    """Infinities and NaN in V of nodes whose scores lie hundreds of powers of two below the cached tokens': they reach every
    row that sees them, and no other one, however the batch cuts the work into runs."""
    T = 20
    c = Case(B, T, hq, hkv, dtype, True, lens, counts=[T] * B, seed=21)
    g = hq // hkv
    c.q.abs_()
    c.k.abs_().mul_(-60)
    clean = c.run().clone()
    inf, nan, two, minus = 3, 5, 7, 9
    c.v[:, inf, :, 5] = math.inf
    c.v[:, nan, :, 70] = math.nan
    c.v[:, two, :, 5] = -math.inf
    c.v[:, minus, :, 127] = -math.inf
    got = c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    plain = [d for d in range(D) if d not in (5, 70, 127)]
    assert torch.equal(got[..., plain], clean[..., plain]) and bool(torch.isfinite(clean).all())
    for b in range(B):
        own = ref.sees(c.parents[b], T, "cuda")
        for d, plus, less in ((5, own[:, inf], own[:, two]), (70, own[:, nan], own[:, nan]),
                              (127, torch.zeros_like(own[:, 0]), own[:, minus])):
            x, y = got[b, :, :, d], clean[b, :, :, d]
            assert torch.equal(x[~plus & ~less], y[~plus & ~less]), (b, d)
            assert bool((x[plus & ~less] == math.inf).all()) and bool((x[~plus & less] == -math.inf).all()), (b, d)
            assert bool(torch.isnan(x[plus & less]).all()), (b, d)
    assert g * hkv == hq


@pytest.mark.parametrize("B,T,lens", [(1, 5, [17]), (2, 200, [3000, 100]), (40, 30, [500] * 40)])
def test_products_end_before_a_call_that_gave_up(monkeypatch, B, T, lens):
    """Values that never arrive: products of scores have been issued in every CTA; the calls end one after another, say so and
    leave NaN, and calls behind them on the same stream are right."""
    c = Case(B, T, 8, 2, "bf16", True, lens, counts=[T] * B)
    want = c.run().clone()
    monkeypatch.setenv("ICE_FAULT", "timeout")
    for _ in range(3):
        c.O.fill_(7)
        c.run()
        assert ice.ice_check(c.err) == ice.ICE_ERR_TIMEOUT and bool(torch.isnan(c.O).all())
    c.run()
    monkeypatch.delenv("ICE_FAULT")
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_TIMEOUT and torch.equal(c.O, want)  # (the error of the call before)
    assert ice.ice_check(c.err) == ice.ICE_OK


@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -20, 2.0 ** -24])
@pytest.mark.parametrize("v_scale", [1.0, 1000.0])
def test_elements_far_below_their_row(small, v_scale):
    """The two halves of V's rows of very different size, element by element, bf16: a row's elements go in as fp16 numbers under
    one power of two f (1 where the row's largest lies in 2^-4 .. 2^8, otherwise the one that brings it to 1 .. 2): off by up
    to 2^-11 of themselves and 2^-24 / f (2^-25 each for a group's mid and for the value)."""
    c = Case(2, 40, 8, 2, "bf16", True, [300, 45], seed=31)
    k, v = ref4.decode(c.recs.view(-1, 2304))
    fine = torch.isfinite(k).all(-1).all(-1) & torch.isfinite(v).all(-1).all(-1)
    half = torch.ones(D, device="cuda")
    half[64:] = small
    new = ref4.encode(torch.nan_to_num(k).bfloat16(), (torch.nan_to_num(v) * half * v_scale).bfloat16())
    c.recs.copy_(torch.where(fine[:, None], new, c.recs.view(-1, 2304)).view_as(c.recs))
    c.v.mul_(half * v_scale)
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    for b in range(c.B):
        n = c.counts[b]
        own = ref.sees(c.parents[b], n, "cuda")
        for j in range(c.hq):
            h = j // 4
            k0, v0 = c.cached(b, h)
            k1, v1 = torch.cat((k0, c.k[b, :n, h].double())), torch.cat((v0, c.v[b, :n, h].double()))
            keep = torch.cat((torch.ones((n, k0.shape[0]), dtype=torch.bool, device="cuda"), own), 1)
            q = c.q[b, :n, j].double()
            w = torch.softmax((q @ k1.T * c.scale).masked_fill(~keep, -math.inf), -1)
            o = w @ v1
            # as tree_ref.tolerance, an element at a time: scores' errors e move it by w e |v - o|, a weight's and a value's
            # own roundings by 2^-11 w |v| each and 2^-24 / f w; weights below 2^-20 of the largest are off by 2^-31 of it
            e = c.scale * 2.0 ** -11 * (q.square() @ k1.square().T).sqrt() + 2.0 ** -22 * (q @ k1.T * c.scale).abs()
            big = v1.abs().amax(-1)  # (7.5 steps beyond mid: at most this, up to the roundings of both)
            up = torch.where((big >= 0.06) & (big <= 250), torch.ones_like(big), 2.0 ** torch.ceil(big.log2()))
            moved = (w * e).square() @ v1.square() + o.square() * (w * e).square().sum(-1, keepdim=True)  # |v - o|^2 <= 2 (..)
            own_err = 2 * 2.0 ** -22 * (w.square() @ v1.square()) + (2.0 ** -24 * w * up).square().sum(-1, keepdim=True)
            tol = 4 * (2 * moved + own_err).sqrt() + 2.0 ** -31 * w.amax(-1, keepdim=True) * v1.abs().sum(0) \
                + (2.0 ** -18 + 2.0 ** -8) * o.abs()
            off = (c.O[b, :n, j].double() - o).abs()
            assert bool((off <= tol).all()), (b, j, float((off / tol).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rest,qs", [(1e-38, 1.0), (1e-38, 1e-4), (1e-38, 1e-30), (1.0, 1.0), (1e30, 1.0)])
def test_a_key_of_minus_infinity_beside_any_others(rest, qs, dtype):
    """A node's key with one element of -inf and others of any size: its score is -inf, so that it weighs nothing with rows that
    see others too, and gives NaN alone."""
    c = Case(2, 6, 8, 2, dtype, True, [40, 0], seed=41, counts=[6, 6])
    c.parents_dev.copy_(torch.tensor([[-1, 0, 1, -1, 3, 2]] * 2, dtype=torch.int32))
    c.parents = [[-1, 0, 1, -1, 3, 2]] * 2
    c.q.abs_().add_(0.01).mul_(qs)
    c.k[:, 1].mul_(rest)
    c.k[:, 1, :, 7] = -math.inf
    c.k[1, 3].mul_(rest)
    c.k[1, 3, :, 100] = -math.inf
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    for b in range(2):
        n = c.counts[b]
        own = ref.sees(c.parents[b], n, "cuda")
        for j in range(c.hq):
            h = j // 4
            k0, v0 = c.cached(b, h)
            k1, v1 = torch.cat((k0, c.k[b, :n, h].double())), torch.cat((v0, c.v[b, :n, h].double()))
            # a node of -inf has no part in anything
            gone = torch.isinf(k1).any(-1)
            keep = torch.cat((torch.ones((n, k0.shape[0]), dtype=torch.bool, device="cuda"), own), 1) & ~gone
            k1[gone] = 0
            alone = ~keep.any(-1)  # (the second sequence's node 3: a root without cached tokens)
            q, got = c.q[b, :n, j].double(), c.O[b, :n, j].double()
            assert bool(torch.isnan(got[alone]).all()) and alone.tolist() == [b == 1 and i == 3 for i in range(n)]
            q, got, keep = q[~alone], got[~alone], keep[~alone]
            want, tol = ref.attention(q, k1, v1, keep, c.scale), ref.tolerance(q, k1, v1, keep, c.scale, c.dt)
            off = (got - want).norm(dim=-1)
            assert bool((off <= tol).all()), (b, j, float((off / tol).max()))
