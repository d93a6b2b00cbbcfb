"""Attention of drafted trees over 4-bit pages, their verification and the commit of what was accepted, against the
64-bit restatements in tree_ref.py and cache4_ref.py."""
import math

import pytest
import torch

import cache4_ref as ref4
import semantic_paged_kv_gb300 as ice
import tree_ref as ref

pytestmark = pytest.mark.gpu
D, S, R = 128, 16, 2304
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _params(B, hq, hkv, dtype, page_cap=1):
    return ice.Config(batch=B, n_q_heads=hq, n_kv_heads=hkv, n_tokens=0, np_cap=1, page_cap=page_cap,
                      dtype=ice.ICE_BF16 if dtype == "bf16" else ice.ICE_FP32).params()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(shape, seed):
    return torch.randn(shape, generator=_gen(seed), device="cuda")


def _records(n, seed, k_scale=1.0, v_scale=1.0):
    k, v = (s * _randn((n, S, D), seed + i) for i, s in enumerate((k_scale, v_scale)))
    return ref4.encode(k.bfloat16(), v.bfloat16())


def _parents(B, T, seed):
    g = torch.Generator().manual_seed(seed)
    p = [[-1] + [int(torch.randint(max(0, (t - 1) // 3), t, (1,), generator=g)) for t in range(1, T)] for _ in range(B)]
    return p, torch.tensor(p, dtype=torch.int32, device="cuda")


class Case:
    """A batch with its cache: ragged lengths, padded trees, pages in any order, garbage (NaN) behind the tokens."""

    def __init__(self, B, T, hq, hkv, dtype, tree, lens, seed=0, k_scale=1.0, v_scale=1.0, q_scale=1.0, counts=None):
        self.B, self.T, self.hq, self.hkv, self.dt = B, T, hq, hkv, DT[dtype]
        self.p = _params(B, hq, hkv, dtype)
        qkv = _randn((B, T, hq + 2 * hkv, D), seed)
        qkv[:, :, :hq] *= q_scale
        qkv[:, :, hq:hq + hkv] *= k_scale
        qkv[:, :, hq + hkv:] *= v_scale
        self.qkv = qkv.to(self.dt)
        self.q, self.k, self.v = self.qkv[:, :, :hq], self.qkv[:, :, hq:hq + hkv], self.qkv[:, :, hq + hkv:]
        self.parents, self.parents_dev = _parents(B, T, seed + 1) if tree else (None, None)
        self.counts = counts or [T if b == 0 else max(0, T - 1 - (3 * b) % (T + 1)) for b in range(B)]
        self.counts_dev = torch.tensor(self.counts, dtype=torch.int32, device="cuda")
        self.tree = ice.Tree(self.parents_dev, self.counts_dev, T)
        self.lens = lens
        self.cache = self.lens_dev = None
        if lens is not None:
            blocks = max(1, -(-max(lens) // S)) + 1
            n = B * blocks + 3
            self.table = torch.randperm(n, generator=_gen(seed + 2), device="cuda")[:B * blocks].view(B, blocks).int()
            self.table = self.table.contiguous()
            self.recs = _records(n * hkv, seed + 3, k_scale, v_scale).view(n, hkv, R)
            # slots behind the last token, and pages nobody has: NaN everywhere
            used = torch.zeros(n, dtype=torch.bool, device="cuda")
            for b, m in enumerate(lens):
                used[self.table[b, :-(-m // S)].long()] = True
                if m % S:
                    self._spoil(int(self.table[b, m // S]), m % S)
            self.recs[~used] = 0xFF
            self.cache = ice.Cache4(self.recs, self.table)
            self.lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.O = torch.full((B, hq, T, D), 7.0, dtype=self.dt, device="cuda").transpose(1, 2)
        self.ws = ice.workspace(ice.ice_tree_workspace_bytes(self.p))
        self.ws.fill_(0xFF)  # no contents are needed
        self.err = _err()
        self.scale = 1 / math.sqrt(D)

    def _spoil(self, page, first):
        at_k, at_v = ref4.places("cuda")
        for t in range(first, S):
            self.recs[page][:, at_k[t]] = 0xFF
            self.recs[page][:, at_v[t]] = 0xFF
            self.recs[page][:, 1024 + 8 * t:1032 + 8 * t] = 0xFF
            self.recs[page][:, 2176 + 8 * t:2184 + 8 * t] = 0xFF

    def run(self, stream=None):
        r = ice.rows
        ice.ice_cache4_attn_tree(self.p, self.tree, r(self.q), self.cache, self.lens_dev, r(self.k), r(self.v),
                                 self.scale, r(self.O), self.ws, self.err, stream)
        return self.O

    def cached(self, b, h):
        """K, V of the cached tokens in 64 bits."""
        m = self.lens[b] if self.lens is not None else 0
        if m == 0:
            return (torch.zeros((0, D), dtype=torch.float64, device="cuda"),) * 2
        k, v = ref4.decode(self.recs[self.table[b, :-(-m // S)].long(), h])
        return k.reshape(-1, D)[:m], v.reshape(-1, D)[:m]

    def each(self, cached=None):
        """(b, head, O64, tolerance) of every head of every sequence with nodes."""
        cached = cached or self.cached
        g = self.hq // self.hkv
        for b in range(self.B):
            n = self.counts[b]
            if n == 0:
                continue
            own = ref.sees(self.parents[b] if self.parents else None, n, "cuda")
            for h in range(self.hkv):
                k0, v0 = cached(b, h)
                k = torch.cat((k0, self.k[b, :n, h].double()))
                v = torch.cat((v0, self.v[b, :n, h].double()))
                keep = torch.cat((torch.ones((n, k0.shape[0]), dtype=torch.bool, device="cuda"), own), 1)
                for j in range(h * g, h * g + g):
                    q = self.q[b, :n, j].double()
                    yield b, j, ref.attention(q, k, v, keep, self.scale), ref.tolerance(q, k, v, keep, self.scale, self.dt)

    def check(self, cached=None):
        for b, j, want, tol in self.each(cached):
            got = self.O[b, :self.counts[b], j].double()
            off = (got - want).norm(dim=-1)
            assert bool((off <= tol).all()), (b, j, float((off / tol).max()))
        for b in range(self.B):
            assert bool((self.O[b, self.counts[b]:] == 7).all())


ATTN = [  # B, T, hq, hkv, tree, lens
    (1, 1, 1, 1, False, None), (1, 1, 4, 1, True, [0]), (2, 1, 8, 8, False, [1, 16]), (2, 5, 32, 8, True, [17, 0]),
    (3, 33, 24, 2, True, [130, 128, 127]), (2, 64, 16, 1, True, [1000, 5]), (1, 256, 4, 2, True, [300]),
    (2, 129, 6, 6, False, [250, 3]), (1, 700, 4, 1, False, [513]), (1, 26, 32, 8, True, [5000]),
    (5, 7, 64, 8, True, [0, 1, 2000, 333, 16]), (1, 8, 16, 1, False, [20000]), (17, 3, 5, 5, True, list(range(0, 850, 50))),
    (2, 255, 2, 2, True, None), (3, 130, 16, 2, False, [129, 0, 4097]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,hq,hkv,tree,lens", ATTN)
def test_attention(B, T, hq, hkv, tree, lens, dtype):
    c = Case(B, T, hq, hkv, dtype, tree, lens)
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_same_bits_every_run(dtype):
    c = Case(4, 21, 32, 8, dtype, True, [3000, 17, 900, 12000])
    first = c.run().clone()
    for _ in range(5):
        c.ws.random_(0, 255)
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("dtype,ks,vs,qs", [("bf16", 1e-30, 1.0, 1.0), ("bf16", 1.0, 1e30, 1.0), ("bf16", 1.0, 1e-30, 1.0),
                                            ("bf16", 1e10, 1e-20, 1e-10), ("bf16", 1e-18, 300.0, 1e18),
                                            ("fp32", 1e10, 1e-20, 1e-10), ("fp32", 1.0, 1e30, 1.0)])
def test_attention_scales(dtype, ks, vs, qs):
    c = Case(2, 9, 8, 2, dtype, True, [200, 33], k_scale=ks, v_scale=vs, q_scale=qs)
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_values_of_very_different_size(dtype):
    """Rows of V from 2^-60 to 2^60 times the others, among pages and nodes: those that weigh next to nothing, and those
    that carry the result."""
    c = Case(2, 12, 8, 2, dtype, True, [300, 40], seed=5)
    big = torch.tensor([2.0 ** ((i * 37) % 121 - 60) for i in range(c.recs.shape[0])], device="cuda")
    k, v = ref4.decode(c.recs.view(-1, R))
    v = (v.view(-1, c.hkv, S, D) * big[:, None, None, None]).view(-1, S, D)
    fine = torch.isfinite(k).all(-1).all(-1) & torch.isfinite(v).all(-1).all(-1)
    new = ref4.encode(torch.nan_to_num(k).bfloat16(), torch.nan_to_num(v).bfloat16())
    c.recs.copy_(torch.where(fine[:, None], new, c.recs.view(-1, R)).view_as(c.recs))
    c.v.mul_(torch.tensor([2.0 ** ((t * 29) % 81 - 40) for t in range(c.T)], device="cuda")[None, :, None, None].to(c.dt))
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_large_scores(dtype):
    """Scores of thousands, rising and falling along the cache: the running maximum moves over and over."""
    c = Case(1, 5, 4, 1, dtype, True, [3000], k_scale=30.0, q_scale=20.0)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_node_infinities_stay_with_those_who_see_them(dtype):
    c = Case(2, 40, 8, 2, dtype, True, [100, 0], counts=[40, 33])
    clean = c.run().clone()
    bad_v, bad_k, bad_q = 7, 11, 13
    c.v[0, bad_v, 0, 5] = math.inf
    c.v[0, bad_v, 0, 9] = math.nan
    c.k[0, bad_k, 1] = math.nan
    c.q[1, bad_q, 3] = math.inf
    got = c.run()
    own = ref.sees(c.parents[0], 40, "cuda")
    sv, sk = own[:, bad_v], own[:, bad_k]
    assert torch.equal(got[0][~sv][:, :4], clean[0][~sv][:, :4])  # heads 0 .. 3 read KV head 0
    seen = got[0][sv][:, :4]
    assert bool((seen[..., 5] == math.inf).all()) and bool(torch.isnan(seen[..., 9]).all())
    other = [d for d in range(D) if d not in (5, 9)]
    assert torch.equal(seen[..., other], clean[0][sv][:, :4][..., other])
    assert torch.equal(got[0][~sk][:, 4:], clean[0][~sk][:, 4:]) and bool(torch.isnan(got[0][sk][:, 4:]).all())
    keep = torch.ones((33, 8), dtype=torch.bool, device="cuda")
    keep[bad_q, 3] = False
    assert torch.equal(got[1, :33][keep], clean[1, :33][keep]) and bool(torch.isnan(got[1, bad_q, 3]).all())
    assert bool((got[1, 33:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_in_the_cache_reaches_its_readers(dtype):
    """A cached token whose V group holds NaN: that half of the heads that read it, and nothing else."""
    c = Case(2, 6, 4, 2, dtype, True, [50, 70])
    clean = c.run().clone()
    page = int(c.table[0, 1])
    c.recs[page, 1, 2176 + 8 * 3:2176 + 8 * 3 + 4] = torch.tensor([0, 0, 0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    got = c.run()
    assert torch.equal(got[1], clean[1]) and torch.equal(got[0, :, :2], clean[0, :, :2])
    assert torch.equal(got[0, :, 2:, 64:], clean[0, :, 2:, 64:]) and bool(torch.isnan(got[0, :, 2:, :64]).all())


def test_attention_conditions_on_the_device():
    c = Case(2, 6, 8, 2, "bf16", True, [100, 90])
    before = c.table.clone()
    c.table[0, 2], c.table[1, 1] = -1, c.recs.shape[0]
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_CAPACITY

    def cached(b, h):  # pages that do not exist are left out
        k, v = ref4.decode(c.recs[before[b, :-(-c.lens[b] // S)].long(), h])
        keep = torch.arange(k.shape[0] * S, device="cuda") < c.lens[b]
        keep &= torch.arange(k.shape[0] * S, device="cuda") // S != (2 if b == 0 else 1)
        return k.reshape(-1, D)[keep], v.reshape(-1, D)[keep]

    c.check(cached)
    c.table.copy_(before)
    c.lens_dev[1] = -3
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_CAPACITY
    c.lens = [100, 0]
    c.check()
    c.lens_dev[1] = 10 ** 6
    c.recs.copy_(_records(c.recs.shape[0] * c.hkv, 77).view_as(c.recs))
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_CAPACITY
    c.lens = [100, c.table.shape[1] * S]
    c.check()
    # a parent that comes later, or below -1, counts as none
    c.lens_dev[1] = c.lens[1]
    c.parents_dev[0, 3], c.parents_dev[0, 2] = 3, -2
    c.parents[0][3] = c.parents[0][2] = -1
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_INVALID_ARG
    c.check()


def test_attention_counts_beyond_the_tree_and_without_counts():
    c = Case(3, 9, 8, 2, "bf16", True, [10, 20, 30], counts=[9, 0, 9])
    c.counts_dev.copy_(torch.tensor([100, -5, 9], dtype=torch.int32))
    c.run()
    c.check()
    c.tree = ice.Tree(c.parents_dev, None, 9)
    c.counts = [9, 9, 9]
    c.run()
    c.check()
    c.tree = ice.Tree(None, c.counts_dev, 0)
    c.run()  # no node: nothing


@pytest.mark.parametrize("dtype,tail,T,tree", [("bf16", None, 9, True), ("bf16", [0, 333], 16, True),
                                               ("bf16", [50, 1], 1, False), ("fp32", [17, 200], 7, True),
                                               ("bf16", [40, 90], 300, False)])
def test_attention_over_selected_pages(dtype, tail, T, tree):
    B, hq, hkv, P = 2, 16, 4, 60
    c = Case(B, T, hq, hkv, dtype, tree, tail, seed=3)
    c.p = _params(B, hq, hkv, dtype, page_cap=P)
    U = B * hkv
    recs = _records(U * P, 50).view(U, P, R)
    page_len = torch.randint(0, S + 1, (U, P), generator=_gen(51), device="cuda").int()
    sel = torch.stack([torch.randperm(P, generator=_gen(60 + u), device="cuda")[:41] for u in range(U)]).int()
    count = torch.tensor([0, 1, 8, 9, 41, 100, -2, 40], dtype=torch.int32, device="cuda")
    sel[3, 4], sel[4, 0] = P, -1
    for u, n in enumerate(count.clamp(0, 41).tolist()):
        sel[u, n:] = -7
    r = ice.rows
    ice.ice_sparse_attn_tree4(c.p, c.tree, r(c.q), recs, page_len, sel, count, c.cache, c.lens_dev, r(c.k), r(c.v),
                              c.scale, r(c.O), c.ws, c.err)
    assert ice.ice_check(c.err) == ice.ICE_ERR_CAPACITY  # the two pages that do not exist

    def cached(b, h):
        u = b * hkv + h
        pages = [x for x in sel[u, :max(0, min(41, int(count[u])))].tolist() if 0 <= x < P]
        k0, v0 = Case.cached(c, b, h)
        if not pages:
            return k0, v0
        k, v = ref4.decode(recs[u, pages])
        keep = (torch.arange(S, device="cuda") < page_len[u, pages][:, None]).reshape(-1)
        return torch.cat((k.reshape(-1, D)[keep], k0)), torch.cat((v.reshape(-1, D)[keep], v0))

    c.check(cached)


def test_attention_agrees_with_the_decode_step():
    """One node, itself in the cache: ice_cache4_attn_decode over the tokens before it and it."""
    B, hq, hkv, n = 2, 16, 4, 500
    c = Case(B, 1, hq, hkv, "bf16", False, [n - 1, n - 1], counts=[1, 1])
    c.run()
    k = torch.empty((B, 1, hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    r = ice.rows
    start = torch.tensor([n - 1, n - 1], dtype=torch.int32, device="cuda")
    ice.ice_cache4_append(c.p, 1, None, r(c.k), r(c.v), None, start, None, None, None, c.cache, c.err)
    ice.ice_cache4_read(c.p, 1, c.cache, start, None, r(k), r(v), c.err)
    c.k.copy_(k)
    c.v.copy_(v)
    c.run()
    O = torch.zeros((B, hq, D), device="cuda")
    ws = ice.workspace(ice.ice_attn4_workspace_bytes(c.p))
    ice.ice_cache4_attn_decode(c.p, c.q[:, 0].contiguous(), c.cache, start + 1, c.scale, O, None, ws, c.err)
    assert ice.ice_check(c.err) == ice.ICE_OK
    for b, j, want, tol in c.each():
        assert float((c.O[b, 0, j].double() - O[b, j].double()).norm()) <= float(tol[0]) + 2.0 ** -18 * float(want.norm())


def test_attention_records_behind_4_gb():
    hkv, T = 4, 5
    n = 500000  # 4.6 GB of records
    c = Case(1, T, 8, hkv, "bf16", True, [64])
    recs = torch.empty((n, hkv, R), dtype=torch.uint8, device="cuda")
    where = torch.tensor([[n - 1, n - 7, 3, n - 100, 5]], dtype=torch.int32, device="cuda")
    recs[where[0].long()] = c.recs[c.table[0, :5].long()]
    c.recs, c.table = recs, where
    c.cache = ice.Cache4(recs, where)
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0])
def test_attention_scale(scale, dtype):
    """No weight by the scores, keys that are far away first, and a softmax of one token."""
    c = Case(2, 11, 8, 2, dtype, True, [300, 17], seed=9)
    c.scale = scale
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_smallest_scales(dtype):
    """Keys and values next to the smallest normal numbers: powers of two of their own up to 2^120."""
    c = Case(2, 9, 8, 2, dtype, True, [200, 33], k_scale=1e-36, v_scale=1e-36, q_scale=1e30)
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [1, 400])
def test_attention_scores_of_minus_infinity(dtype, B):
    """A node that sees itself alone, with a score of -inf: NaN there, and nowhere else."""
    c = Case(B, 3, 4, 2, dtype, True, [0] * B, counts=[3] * B)
    c.parents_dev.copy_(torch.tensor([[-1, 0, -1]] * B, dtype=torch.int32))
    c.parents = [[-1, 0, -1]] * B
    c.k[:, 2, :, 0] = -math.inf
    c.q[:, 2, :, 0] = 1.0
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    assert bool(torch.isnan(c.O[:, 2]).all()) and bool(torch.isfinite(c.O[:, :2]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_in_place(dtype):
    """O over q, in a projection's layout: the same bits."""
    c = Case(2, 40, 16, 4, dtype, True, [700, 0], counts=[40, 22])
    want = c.run().clone()
    before = c.q.clone()
    c.O = c.q
    c.run()
    for b in range(2):
        n = c.counts[b]
        assert torch.equal(c.q[b, :n], want[b, :n]) and torch.equal(c.q[b, n:], before[b, n:])


def test_attention_long_chain():
    """A chunk of 3001 tokens behind 40: rows of many blocks, some before and some behind each tile's nodes."""
    c = Case(1, 3001, 2, 1, "bf16", False, [40])
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,hq,hkv,tree,lens", [
    (13, 500, 32, 2, False, None), (40, 300, 16, 1, False, None), (30, 40, 32, 8, True, [0] * 20 + [300, 0, 0, 0, 2000] * 2),
    (24, 200, 16, 2, True, [0, 0, 0, 0, 0, 300] * 4), (60, 9, 16, 4, True, [0] * 40 + [129, 257] * 10)])
def test_attention_short_segments_before_longer_ones(B, T, hq, hkv, tree, lens, dtype):
    """Many blocks of one tile, then blocks of several, in one CTA's run: warps that have no part in the short ones wait for
    them all the same."""
    c = Case(B, T, hq, hkv, dtype, tree, lens, counts=[T - b % 3 for b in range(B)])
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


def test_attention_many_units():
    """More units than a CTA has threads, most of one or two tiles."""
    c = Case(40, 2, 32, 32, "bf16", True, [(37 * b) % 90 for b in range(40)])
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


def test_attention_wait_that_gives_up(monkeypatch):
    """Pages that never arrive: the waits end, the call says so and leaves NaN, and the next call is right."""
    c = Case(2, 9, 8, 2, "bf16", True, [3000, 100])
    monkeypatch.setenv("ICE_FAULT", "timeout")
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_ERR_TIMEOUT
    for b in range(2):
        assert bool(torch.isnan(c.O[b, :c.counts[b]]).all()) and bool((c.O[b, c.counts[b]:] == 7).all())
    monkeypatch.delenv("ICE_FAULT")
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()


def test_attention_workspace_between_shapes_and_graphs():
    """One workspace for calls of different shapes one after another, eager and captured."""
    cases = [Case(1, 26, 32, 8, "bf16", True, [5000]), Case(4, 7, 8, 2, "fp32", True, [300, 1, 0, 77]),
             Case(2, 200, 16, 4, "bf16", False, [100, 2000])]
    want = [c.run().clone() for c in cases]
    for c in cases:
        c.ws = cases[0].ws
    graphs = []
    for c in cases:
        c.O.fill_(7)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for _ in range(2):
        for c, g, w in zip(cases, graphs, want):
            c.O.fill_(7)
            g.replay()
            cases[1].run()
            assert torch.equal(c.O, w) and torch.equal(cases[1].O, want[1])


def test_attention_on_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    cases = [Case(2, 40, 16, 4, "bf16", True, [3000, 70]), Case(9, 5, 8, 8, "bf16", False, [900] * 9),
             Case(2, 12, 8, 2, "fp32", True, [500, 40])]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert ice.ice_check(c.err) == ice.ICE_OK and torch.equal(c.O, w)


# ----------------------------------------------------------------- verify --
def _verify(target, draft, tokens, parents, counts, uniform):
    B, T = tokens.shape
    path = torch.full((B, T), 99, dtype=torch.int32, device="cuda")
    n, nxt = torch.full((B,), 99, dtype=torch.int32, device="cuda"), torch.full((B,), 99, dtype=torch.int32, device="cuda")
    err = _err()
    ice.ice_tree_verify(ice.Tree(parents, counts, T), ice.probs(target), None if draft is None else ice.probs(draft),
                        tokens, uniform, path, n, nxt, err)
    return path, n, nxt, ice.ice_check(err)


def _check_verify(target, draft, tokens, parents, counts, uniform, status=ice.ICE_OK, near_ok=0):
    path, n, nxt, got = _verify(target, draft, tokens, parents, counts, uniform)
    assert got == status
    B, T = tokens.shape
    skipped = 0
    for b in range(B):
        m = T if counts is None else max(0, min(T, int(counts[b])))
        want, x, near = ref.verify(target[b].double().cpu(), None if draft is None else draft[b].double().cpu(),
                                   tokens[b].tolist(), None if parents is None else parents[b].tolist(),
                                   None if uniform is None else uniform[b].double().tolist(), m)
        if near < 1e-11:  # sums in another order may decide otherwise
            skipped += 1
            continue
        assert path[b].tolist() == want + [-1] * (T - len(want)), b
        assert int(n[b]) == len(want) and int(nxt[b]) == x, b
    assert skipped <= near_ok


def _probs(B, T, V, dtype, seed, peak=3.0, noise=0.7):
    z = peak * _randn((B, T, V), seed)
    return torch.softmax(z, -1).to(DT[dtype]), torch.softmax(z + noise * _randn((B, T, V), seed + 1), -1).to(DT[dtype])


def _tokens(draft, parents, seed):
    up = torch.tensor([[max(0, x) for x in p] for p in parents], device="cuda")
    q = draft.float().gather(1, up[..., None].expand(*up.shape, draft.shape[-1]))
    noise = torch.empty_like(q).exponential_(generator=_gen(seed))
    return (q / noise).argmax(-1).int()


VERIFY = [(1, 1, 1), (2, 2, 7), (3, 9, 50), (33, 26, 1000), (4, 61, 4099), (2, 130, 333), (1, 1024, 64), (2, 5, 128000),
          (3, 17, 32003)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["sample", "certain", "greedy"])
@pytest.mark.parametrize("B,T,V", VERIFY)
def test_verify(B, T, V, mode, dtype):
    target, draft = _probs(B, T, V, dtype, 3)
    parents, dev = _parents(B, T, 4)
    tokens = _tokens(draft, parents, 5)
    if mode == "greedy":  # some of them the target's likeliest
        best = torch.stack([target[b].argmax(-1)[[max(0, x) for x in parents[b]]] for b in range(B)]).int()
        tokens = torch.where(torch.rand((B, T), generator=_gen(6), device="cuda") < 0.5, best, tokens)
    uniform = torch.rand((B, T), generator=_gen(7), device="cuda") if mode != "greedy" else None
    counts = torch.tensor([T if b % 3 == 0 else (b * 7) % (T + 1) for b in range(B)], dtype=torch.int32, device="cuda")
    _check_verify(target, draft if mode == "sample" else None, tokens, dev, counts, uniform)
    # a chain, every node there
    _check_verify(target, draft if mode == "sample" else None, tokens, None, None, uniform)


def test_verify_many_refusals():
    """A wide node whose children are nearly all refused: the same token again and again, a draft far from the target."""
    B, T, V = 8, 100, 257
    target, draft = _probs(B, T, V, "fp32", 11, peak=2.0, noise=6.0)
    parents = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    parents[:, 0] = -1
    tokens = _tokens(draft, parents.tolist(), 12)
    tokens[:, 10:20] = tokens[:, 9:10]
    uniform = torch.rand((B, T), generator=_gen(13), device="cuda")
    uniform[:4, 1:] = 0.999
    _check_verify(target, draft, tokens, parents, None, uniform)
    _check_verify(target, None, tokens, parents, None, uniform)


def test_verify_strided_and_unaligned_rows():
    B, T, V = 3, 11, 997
    t, d = _probs(B, T, V, "bf16", 21)
    big_t = torch.zeros((B, T, V + 5), dtype=torch.bfloat16, device="cuda")
    big_t[..., 3:V + 3] = t
    big_d = torch.zeros((T, B, V + 2), dtype=torch.bfloat16, device="cuda")
    big_d[..., 1:V + 1] = d.transpose(0, 1)
    parents, dev = _parents(B, T, 22)
    tokens = _tokens(d, parents, 23)
    uniform = torch.rand((B, T), generator=_gen(24), device="cuda")
    _check_verify(big_t[..., 3:V + 3], big_d[..., 1:V + 1].transpose(0, 1), tokens, dev, None, uniform)
    # one distribution for every node: stride 0
    _check_verify(t[:, :1].expand(B, T, V), d, tokens, dev, None, uniform)


@pytest.mark.parametrize("u", [0.0, 0.5, 1 - 2.0 ** -24])
def test_verify_borders(u):
    """Probabilities that are multiples of 2^-6 (every sum is exact): decisions on their borders."""
    V, T = 64, 4
    target = torch.zeros((1, T, V), device="cuda")
    draft = torch.zeros((1, T, V), device="cuda")
    target[0, :, 3], target[0, :, 10], target[0, :, 63] = 0.5, 0.25, 0.25
    draft[0, :, 10], draft[0, :, 20] = 0.5, 0.5
    tokens = torch.tensor([[0, 10, 20, 3]], dtype=torch.int32, device="cuda")
    for parents in (None, torch.tensor([[-1, 0, 0, 0]], dtype=torch.int32, device="cuda")):
        uniform = torch.full((1, T), u, device="cuda")
        for dr in (draft, None, target):
            path, n, nxt, err = _verify(target, dr, tokens, parents, None, uniform)
            want, x, _ = ref.verify(target[0].double().cpu(), None if dr is None else dr[0].double().cpu(),
                                    tokens[0].tolist(), None if parents is None else parents[0].tolist(),
                                    uniform[0].double().tolist(), T)
            assert err == ice.ICE_OK and path[0].tolist() == want + [-1] * (T - len(want)) and int(nxt[0]) == x


def test_verify_odd_inputs():
    B, T, V = 6, 5, 40
    target, draft = _probs(B, T, V, "fp32", 31)
    parents = torch.tensor([[-1, 0, 0, 1, 2]] * B, dtype=torch.int32, device="cuda")
    tokens = _tokens(draft, parents.tolist(), 32)
    uniform = torch.rand((B, T), generator=_gen(33), device="cuda")
    # a row without any probability
    z = target.clone()
    z[2] = 0
    path, n, nxt, err = _verify(z, None, tokens, parents, None, uniform)
    assert err == ice.ICE_ERR_INVALID_ARG and int(nxt[2]) == -1 and path[2].tolist() == [0, -1, -1, -1, -1]
    # NaN and negative probabilities count as nothing
    z = target.clone()
    z[..., 7], z[..., 8] = math.nan, -0.5
    for mode in ("sample", "certain", "greedy"):
        _check_verify(z, draft if mode == "sample" else None, tokens, parents, None, None if mode == "greedy" else uniform)
    z = torch.full_like(target, math.nan)
    path, n, nxt, err = _verify(z, None, tokens, parents, None, None)
    assert err == ice.ICE_ERR_INVALID_ARG and bool((nxt == -1).all()) and bool((n == 1).all())
    # tokens outside the vocabulary are never accepted
    bad = tokens.clone()
    bad[:, 1], bad[:, 3] = V, -1
    for u in (uniform, None):
        _check_verify(target, draft if u is not None else None, bad, parents, None, u, ice.ICE_ERR_CAPACITY)
    # a second root is not reached; a parent that comes later counts as one
    par = parents.clone()
    par[:, 1] = -1
    _check_verify(target, draft, tokens, par, None, uniform)
    par[:, 1] = 4
    path, n, nxt, err = _verify(target, draft, tokens, par, None, uniform)
    assert err == ice.ICE_ERR_INVALID_ARG
    par[:, 1] = -1
    want = _verify(target, draft, tokens, par, None, uniform)
    assert torch.equal(path, want[0]) and torch.equal(nxt, want[2])
    # node 0's token and parent are not read
    tokens[:, 0] = 10 ** 9
    _check_verify(target, draft, tokens, parents, None, uniform)


def test_verify_keeps_the_target_distribution():
    """20000 trees of one node with three children drawn from the draft: the first token behind the root is distributed
    as the target's (each frequency within 5 standard deviations)."""
    B, T, V = 20000, 4, 12
    p = torch.softmax(1.5 * _randn((V,), 41), -1)
    q = torch.softmax(1.5 * _randn((V,), 42), -1)
    target, draft = (x.expand(B, T, V) for x in (p, q))
    parents = torch.tensor([[-1, 0, 0, 0]], dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    tokens = torch.multinomial(q.expand(B, V), T, replacement=True, generator=_gen(43)).int()
    uniform = torch.rand((B, T), generator=_gen(44), device="cuda")
    path, n, nxt, err = _verify(target, draft, tokens, parents, None, uniform)
    assert err == ice.ICE_OK
    first = torch.where(n > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    freq = torch.bincount(first.long(), minlength=V).double().cpu() / B
    p = p.double().cpu()
    assert bool(((freq - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all())
    # the first child alone is accepted with probability sum min(p, q)
    least = float(torch.minimum(p, q.double().cpu()).sum())
    assert float((n > 1).double().mean()) >= least - 5 * (least * (1 - least) / B) ** 0.5


# ----------------------------------------------------------------- commit --
@pytest.mark.parametrize("dtype,L,B,T,hkv", [("bf16", 1, 1, 1, 1), ("bf16", 3, 2, 26, 8), ("fp32", 2, 3, 7, 3),
                                             ("bf16", 1, 2, 300, 5), ("bf16", 40, 16, 9, 2), ("fp32", 1, 1, 64, 32)])
def test_commit(dtype, L, B, T, hkv):
    p = _params(B, hkv, hkv, dtype)
    kv = _randn((2, B, L, T, hkv, D), 1).to(DT[dtype])  # layers inside the batch: strides of any order
    k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    start = [(b * 13) % 40 for b in range(B)]
    n = [min(T, (1, 0, 5, T, 17)[(b + (T > 200)) % 5] if b or T > 200 else T) for b in range(B)]
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        path[b, :n[b]] = torch.randperm(T, generator=_gen(b), device="cuda")[:n[b]].sort().values.int()
    blocks = (max(start) + T) // S + 1
    pages = B * blocks + 1
    table = torch.randperm(pages, generator=_gen(9), device="cuda")[:B * blocks].view(B, blocks).int().contiguous()
    recs = torch.full((L, pages + 1, hkv, R), 0xAB, dtype=torch.uint8, device="cuda")
    want = recs.clone()
    at_k, at_v = ref4.places("cuda")
    for b in range(B):
        for i in range(n[b]):
            t = start[b] + i
            page, s = int(table[b, t // S]), t % S
            row = torch.zeros((2, L * hkv, S, D), dtype=DT[dtype], device="cuda")
            row[0, :, s] = k[:, b, int(path[b, i])].reshape(-1, D)
            row[1, :, s] = v[:, b, int(path[b, i])].reshape(-1, D)
            rec = ref4.encode(row[0], row[1]).view(L, hkv, R)
            for cols in (at_k[s], at_v[s], torch.arange(1024 + 8 * s, 1032 + 8 * s, device="cuda"),
                         torch.arange(2176 + 8 * s, 2184 + 8 * s, device="cuda")):
                want[:, page][..., cols] = rec[..., cols]
    err = _err()
    start_dev = torch.tensor(start, dtype=torch.int32, device="cuda")
    n_dev = torch.tensor([x if x != T else T + 5 * (b % 2) for b, x in enumerate(n)], dtype=torch.int32, device="cuda")
    ice.ice_cache4_commit(p, L, T, ice.rows(k[0]), ice.rows(v[0]), path, n_dev, start_dev,
                          ice.Cache4(recs[0, :pages], table), err, k_layer=k.stride(0), v_layer=v.stride(0),
                          records_layer=recs.stride(0))
    assert ice.ice_check(err) == ice.ICE_OK
    assert torch.equal(recs, want)
    assert start_dev.tolist() == start


def test_commit_outside_the_cache():
    B, T, hkv = 3, 6, 2
    p = _params(B, hkv, hkv, "bf16")
    k, v = _randn((B, T, hkv, D), 1).bfloat16(), _randn((B, T, hkv, D), 2).bfloat16()
    table = torch.arange(B * 2, dtype=torch.int32, device="cuda").view(B, 2)
    recs = torch.full((B * 2, hkv, R), 0xAB, dtype=torch.uint8, device="cuda")
    path = torch.tensor([[0, 6, 2, -1, 3, 4], [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5]], dtype=torch.int32, device="cuda")
    n = torch.tensor([6, 4, 3], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 30, -1], dtype=torch.int32, device="cuda")
    err = _err()
    ice.ice_cache4_commit(p, 1, T, ice.rows(k), ice.rows(v), path, n, start, ice.Cache4(recs, table), err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    ko, vo = (torch.full((B, T, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ice.ice_cache4_read(p, T, ice.Cache4(recs, table), torch.tensor([0, 30, 0], dtype=torch.int32, device="cuda"),
                        torch.tensor([6, 2, 2], dtype=torch.int32, device="cuda"), ice.rows(ko), ice.rows(vo), err)
    held = lambda x: ref4.held(x).bfloat16()  # noqa: E731
    for i, node in ((0, 0), (2, 2), (4, 3), (5, 4)):
        assert torch.equal(ko[0, i], held(k[0, node])) and torch.equal(vo[0, i], held(v[0, node]))
    assert torch.equal(ko[1, :2], held(k[1, :2])) and torch.equal(ko[2, :2], held(k[2, 1:3]))
    raw = recs.view(B, 2, hkv, R)
    at_k, _ = ref4.places("cuda")
    for i in (1, 3, 6):  # the slots that were left out, and the next one
        assert bool((raw[0, 0][:, at_k[i]] == 0xAB).all())


# --------------------------------------------------------------- together --
class Step:
    """Speculative steps of a small model's layers: rotation, attention of the tree, verification and commit."""

    def __init__(self, L=3, B=2, T=9, hq=8, hkv=2, V=50, start=(40, 7)):
        self.L, self.B, self.T, self.hq, self.hkv, self.V = L, B, T, hq, hkv, V
        self.p = _params(B, hq, hkv, "bf16")
        blocks = (max(start) + 4 * T) // S + 2
        self.table = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
        self.recs = _records(L * B * blocks * hkv, 7).view(L, B * blocks, hkv, R)
        self.caches = [ice.Cache4(self.recs[i], self.table) for i in range(L)]
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        inv = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        table = torch.empty((4000, D // 2, 2), device="cuda")
        ice.ice_rope_table(inv, 4000, table)
        self.rope = ice.Rope(table)
        self.parents, self.parents_dev = _parents(B, T, 3)
        depth = torch.tensor([[len(self._up(b, t)) for t in range(T)] for b in range(B)], dtype=torch.int32, device="cuda")
        self.depth = depth
        self.tree = ice.Tree(self.parents_dev)
        self.qkv = torch.zeros((L, B, T, hq + 2 * hkv, D), dtype=torch.bfloat16, device="cuda")
        self.q, self.k, self.v = (torch.zeros((L, B, T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
        self.O = torch.zeros_like(self.q)
        self.target, self.draft = (torch.zeros((B, T, V), device="cuda") for _ in range(2))
        self.tokens = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        self.uniform = torch.zeros((B, T), device="cuda")
        self.path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        self.n, self.next = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        self.positions = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        self.ws = ice.workspace(ice.ice_tree_workspace_bytes(self.p))
        self.err = _err()

    def _up(self, b, t):
        out = []
        while self.parents[b][t] >= 0:
            t = self.parents[b][t]
            out.append(t)
        return out

    def fill(self, seed):
        self.qkv.copy_(_randn(self.qkv.shape, seed).bfloat16())
        t, d = _probs(self.B, self.T, self.V, "fp32", seed + 1)
        self.target.copy_(t)
        self.draft.copy_(d)
        self.tokens.copy_(_tokens(d, self.parents, seed + 2))
        self.uniform.copy_(torch.rand(self.uniform.shape, generator=_gen(seed + 3), device="cuda"))

    def run(self):
        r, hq, hkv = ice.rows, self.hq, self.hkv
        torch.add(self.start[:, None], self.depth, out=self.positions)
        for i in range(self.L):
            x = self.qkv[i]
            ice.ice_qkv_rope(self.p, self.T, r(x[:, :, :hq]), r(x[:, :, hq:hq + hkv]), r(x[:, :, hq + hkv:]),
                             self.positions, None, None, self.rope, r(self.q[i]), r(self.k[i]), r(self.v[i]), self.err)
            ice.ice_cache4_attn_tree(self.p, self.tree, r(self.q[i]), self.caches[i], self.start, r(self.k[i]),
                                     r(self.v[i]), 1 / math.sqrt(D), r(self.O[i]), self.ws, self.err)
        ice.ice_tree_verify(self.tree, ice.probs(self.target), ice.probs(self.draft), self.tokens, self.uniform,
                            self.path, self.n, self.next, self.err)
        ice.ice_cache4_commit(self.p, self.L, self.T, r(self.k[0]), r(self.v[0]), self.path, self.n, self.start,
                              self.caches[0], self.err, k_layer=self.k.stride(0), v_layer=self.v.stride(0),
                              records_layer=self.recs.stride(0))
        self.start += self.n

    def state(self):
        return [x.clone() for x in (self.O, self.path, self.n, self.next, self.start, self.recs)]


def test_steps_as_appended_one_by_one():
    """Two speculative steps leave the caches that ice_cache4_append of the accepted tokens alone leaves."""
    s = Step()
    recs, start = s.recs.clone(), s.start.clone()
    for seed in (100, 200):
        s.fill(seed)
        s.run()
        for b in range(s.B):
            n = int(s.n[b])
            at = s.path[b, :n].long()
            p1 = _params(1, s.hq, s.hkv, "bf16")
            for i in range(s.L):
                x = s.qkv[i, b:b + 1, at]
                k, v = (ice.rows(y.contiguous()) for y in (x[:, :, s.hq:s.hq + s.hkv], x[:, :, s.hq + s.hkv:]))
                ice.ice_cache4_append(p1, n, None, k, v, None, start[b:b + 1].clone(), None, s.rope, None,
                                      ice.Cache4(recs[i], s.table[b:b + 1].contiguous()), s.err)
            start[b] += n
    assert ice.ice_check(s.err) == ice.ICE_OK
    assert torch.equal(s.start, start) and torch.equal(s.recs, recs) and bool((s.n >= 1).all())


def test_steps_in_a_graph_and_on_other_streams():
    a, b = Step(), Step()
    graph_of = Step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph_of.fill(1)
    keep = graph_of.state()
    with torch.cuda.stream(side):
        graph_of.run()
    torch.cuda.current_stream().wait_stream(side)
    graph_of.recs.copy_(keep[5])
    graph_of.start.copy_(keep[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_of.run()
    graph_of.recs.copy_(keep[5])
    graph_of.start.copy_(keep[4])
    for seed in (10, 20, 30):
        for x in (a, b, graph_of):
            x.fill(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # two steps of workspaces of their own at once
            b.run()
        a.run()
        graph.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(a.state(), b.state(), graph_of.state()):
            assert torch.equal(x, y) and torch.equal(x, z)
    assert ice.ice_check(a.err) == ice.ICE_OK
