"""The operators of the 4-bit pages where their number ranges end, where heads and tokens of one call differ in size,
and over more units than a CTA keeps at hand, against the 64-bit restatement in cache4_ref.py."""
import math

import pytest
import torch

import cache4_ref as ref
import semantic_paged_kv_gb300 as ice
from test_gpu_cache4 import (D, DT, R, S, _attn_buffers, _cache, _err, _gen, _ix, _params, _poison, _qkv,
                             _random_records, _rows_of, _table)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- quantiser --
def _pack(k, v, dtype):
    """Records and the values read back of pages k, v [n, 16, 128]."""
    n = k.shape[0]
    p = _params(1, 1, 1, dtype, page_cap=n)
    lens = torch.full((1, n), S, dtype=torch.int32, device="cuda")
    cnt = torch.full((1,), n, dtype=torch.int32, device="cuda")
    recs, err = torch.empty((1, n, R), dtype=torch.uint8, device="cuda"), _err()
    ice.ice_pool4_pack(p, _ix(n_pages=cnt, page_len=lens, pool_k=k, pool_v=v), 0, recs, err)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    ice.ice_pool4_unpack(p, _ix(n_pages=cnt, page_len=lens, pool_k=ko, pool_v=vo), recs, err)
    assert ice.ice_check(err) == ice.ICE_OK
    return recs[0], ko, vo


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_groups_at_the_top_of_the_range(dtype):
    """Extremes whose sum overflows fp32 while their difference does not: mid is finite, and so is what the group
    stands for."""
    n, g = 64, _gen(201)
    big = float(torch.finfo(torch.bfloat16).max)
    x = torch.rand((n, S, D), generator=g, device="cuda") * 1.5e38 + 1.8e38  # 1.8e38 .. 3.3e38
    x[1] = x[1].sign() * 3e38
    x[2] = big
    x[3] = 3.3e38 + torch.rand((S, D), generator=g, device="cuda") * 4e36  # a narrow group beside the largest value
    x[4, :, ::3] = 1e38
    x[5, :, 1::2] = 2.0 ** 127
    x[6] = 1.7e38 + torch.rand((S, D), generator=g, device="cuda") * 1e37  # sums on either side of the overflow
    x[:, 8:] *= -1
    k = x.to(DT[dtype]).clamp(-big, big)
    if dtype == "fp32":  # mid rounds up, so that mid + 7 step lies beyond fp32's largest value
        k[7] = torch.linspace(3.31244e38, torch.finfo(torch.float32).max, D, device="cuda")[torch.randperm(D, generator=g,
                                                                                                        device="cuda")]
        k[7, :, 0], k[7, :, 1], k[7, :, 64], k[7, :, 65] = k[7].amax(), k[7].amin(), k[7].amax(), k[7].amin()
    v = k.flip(1).contiguous()
    recs, ko, vo = _pack(k, v, dtype)
    assert torch.equal(recs, ref.encode(k, v))
    for o, y in ((ko, k), (vo, v)):
        assert torch.equal(o, ref.held(y).float().to(DT[dtype]))
    assert bool(ko[1].isfinite().all()) and bool((ko[1].float().abs() > 2.9e38).all()) and torch.equal(ko[2], k[2])


def test_lowest_fp32_value():
    """fp32 values beyond the largest bf16 number: mid rounds to infinity, as bf16((max + min) / 2) does."""
    k = torch.full((1, S, D), torch.finfo(torch.float32).min, device="cuda")
    v = -k
    recs, ko, vo = _pack(k, v, "fp32")
    assert torch.equal(recs, ref.encode(k, v)) and bool((ko == -math.inf).all()) and bool((vo == math.inf).all())


def test_codes_of_tiny_values_beside_large_ones():
    """x - mid does not fit fp32: the code of a tiny value hangs on its sign where mid lies on a border."""
    n, g = 2000, _gen(202)
    x = torch.randint(-13, 18, (n, S, D), generator=g, device="cuda").float()
    x[..., 0::64], x[..., 1::64] = 17, -13  # step 2, mid 2: 0 lies half a step from two codes
    tiny = torch.exp2(torch.randint(-80, -15, (n, S, D), generator=g, device="cuda").float())
    tiny *= torch.randint(-1, 2, (n, S, D), generator=g, device="cuda")
    at = torch.arange(D, device="cuda") % 4 == 2
    x = torch.where(at, tiny, x)
    x[0, 0, 2] = 3e-8
    x[n // 2:] *= torch.exp2(torch.randint(-60, 60, (n - n // 2, S, 1), generator=g, device="cuda").float())
    k = x.bfloat16()
    v = k.flip(-1).contiguous()
    recs, _, _ = _pack(k, v, "bf16")
    meta, codes = ref.groups(k)
    assert meta[0, 0, 0].tolist() == [2.0, 2.0] and int(codes[0, 0, 2]) == 7
    assert torch.equal(recs, ref.encode(k, v))


def test_steps_of_tiny_fp32_groups():
    """Extremes below 1e-30 whose difference is rounded in fp32: the step is that of the difference itself (pairs whose
    rounded difference leads to the other neighbour in bf16, and random ones)."""
    pairs = [(-2.33786149e-31, 1.69214669e-31), (-6.59842301e-33, 6.44674383e-33), (-8.90160388e-37, 1.06593559e-36),
             (-3.16460062e-36, 3.38143391e-36), (-6.64765244e-34, 4.04464372e-34), (-3.024296e-32, 3.16877219e-32),
             (-2.35131282e-36, 1.27435275e-36), (-2.08655305e-36, 1.38482852e-36), (-2.33794003e-34, 1.76688602e-34),
             (-5.57138979e-35, 3.36824447e-35), (-1.77763456e-34, 1.4173592e-34), (-2.41923673e-31, 2.15966195e-31)]
    n, g = 200, _gen(204)
    x = torch.rand((n, S, D), generator=g, device="cuda") * 2 - 1
    x *= torch.exp2(torch.randint(-149, -95, (n, S, 1), generator=g, device="cuda").float())
    for i, (lo, hi) in enumerate(pairs):
        x[i, :, :] = torch.rand((S, D), generator=g, device="cuda") * lo
        x[i, :, 5::64], x[i, :, 40::64] = lo, hi
    x = torch.where(x == 0, torch.zeros_like(x), x)
    k, v = x.contiguous(), x.flip(0).contiguous()
    recs, _, _ = _pack(k, v, "fp32")
    assert torch.equal(recs, ref.encode(k, v))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_codes_of_negative_zeros(dtype):
    """-0.0 halfway between two codes has the code of 0.0 (values pruned to zero keep their signs)."""
    n, g = 500, _gen(203)
    x = (torch.randn((n, S, D), generator=g, device="cuda") * 4).round() / 4
    x[..., 0::64], x[..., 1::64] = 3, -3  # mid 0
    x = torch.where(torch.rand((n, S, D), generator=g, device="cuda") < 0.3, torch.zeros_like(x), x)
    x[..., 0::64], x[..., 1::64] = 3, -3
    minus = torch.where(x == 0, -torch.zeros_like(x), x)
    assert bool(torch.signbit(minus[x == 0]).all())
    plus = _pack(x.to(DT[dtype]), x.flip(0).contiguous().to(DT[dtype]), dtype)[0]
    recs = _pack(minus.to(DT[dtype]), minus.flip(0).contiguous().to(DT[dtype]), dtype)[0]
    assert torch.equal(recs, plus)
    assert torch.equal(recs, ref.encode(x.to(DT[dtype]), x.flip(0).to(DT[dtype])))


# ------------------------------------------------------ append: the norm --
def _normed(x, w, eps):
    """Norm of keys as ice.h states it, an fp32 rounding at each step, the sum of squares rounded once."""
    ms = x.double().square().sum(-1, keepdim=True).float() / D
    r = (1 / (ms + torch.tensor(eps, dtype=torch.float32, device="cuda")).double().sqrt()).float()
    return (x.float() * r) * w.float()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_of_keys_to_the_last_bit(dtype):
    """Keys after the norm alone: the error-free sum of squares leaves no rounding but its own."""
    B, T, hkv = 1, 3000, 2
    x = torch.randn((B, T, hkv, D), generator=_gen(211), device="cuda")
    x *= torch.exp2(torch.randint(-3, 4, x.shape, generator=_gen(212), device="cuda").float())
    k = x.to(DT[dtype])
    w = (1 + 0.3 * torch.randn(D, generator=_gen(213), device="cuda")).to(DT[dtype])
    out, err = torch.empty_like(k), _err()
    ice.ice_qkv_rope(_params(B, hkv, hkv, dtype), T, None, ice.rows(k), None, None, None, None,
                     ice.Rope(None, k_norm=w, eps=1e-6), None, ice.rows(out), None, err)
    assert ice.ice_check(err) == ice.ICE_OK
    assert torch.equal(out, _normed(k, w, 1e-6).to(DT[dtype]))


@pytest.mark.parametrize("dtype,rd,inter,norm", [("bf16", 128, False, True), ("bf16", 64, True, True),
                                                 ("bf16", 128, False, False), ("fp32", 128, False, True),
                                                 ("fp32", 96, True, True), ("fp32", 128, False, False)])
def test_append_at_positions_unlike_the_slots(dtype, rd, inter, norm):
    """The tail behind an index: cache slots from 0, rotation positions behind the prompt, any order; norms in fp32
    too.  The records against the restatement."""
    B, T, hq, hkv = 3, 45, 4, 2
    p = _params(B, hq, hkv, dtype)
    _, q, k, v = _qkv(B, T, hq, hkv, dtype, 221, 3.0)
    table = _table(rd, 120000)[1]
    pos = torch.randint(0, 120000, (B, T), generator=_gen(222), device="cuda").int()
    w = (1 + 0.3 * torch.randn(D, generator=_gen(223), device="cuda")).to(DT[dtype])
    rope = ice.Rope(table, interleaved=inter, q_norm=w if norm else None, k_norm=w if norm else None)
    start = torch.tensor([0, 3, 16], dtype=torch.int32, device="cuda")
    blocks = 5
    recs, bt = _cache(B, blocks, hkv, 224)
    qo, err, r = torch.empty((B, T, hq, D), dtype=DT[dtype], device="cuda"), _err(), ice.rows
    ice.ice_cache4_append(p, T, r(q), r(k), r(v), pos, start, None, rope, r(qo), ice.Cache4(recs, bt), err)
    assert ice.ice_check(err) == ice.ICE_OK
    y = _normed(k, w, 1e-6) if norm else k.float()
    cs = table[pos.long()]
    if dtype == "fp32":  # products and their sum before one rounding
        y = ref.rotate(y, cs, inter).float()
    else:  # each product and their sum rounded to fp32, then to bf16
        c, s = cs[..., None, :, 0], cs[..., None, :, 1]
        z = y.clone()
        a, b = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, rd // 2), slice(rd // 2, rd))
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        y = z.to(DT[dtype])
    K, V = _rows_of(recs, bt, 0)
    for b in range(B):
        a = int(start[b])
        assert torch.equal(K[b, :, a:a + T], ref.held(y[b]).transpose(0, 1))
        assert torch.equal(V[b, :, a:a + T], ref.held(v[b]).transpose(0, 1))
    # the queries at those positions, relative to 64 bits: norm and rotation round at most 8 times in fp32
    want = ref.rotate(ref.norm(q, w, 1e-6) if norm else q.double(), cs, inter)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = half * want.abs() + 8 * 2.0 ** -24 * 2 * want.abs().amax(-1, keepdim=True)
    assert bool(((qo.double() - want).abs() <= tol).all())


def test_pack_of_many_inserted_tokens():
    """Only the tokens from first_token on, hundreds of them a unit: the records of a whole pack."""
    B, hq, hkv, N, first = 2, 6, 3, 900, 123
    cfg = ice.Config(batch=B, n_q_heads=hq, n_kv_heads=hkv, n_tokens=N, seed=5)
    p = cfg.params()
    K, V = (torch.randn((B, hkv, N, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    idx, err = ice.Index(cfg), _err()
    ice.ice_build_index(p, K, V, idx, ice.workspace(ice.ice_build_workspace_bytes(p)), err)
    whole = torch.zeros(ice.ice_pool4_bytes(p), dtype=torch.uint8, device="cuda").view(cfg.units, cfg.page_cap, R)
    part = torch.zeros_like(whole)
    ice.ice_pool4_pack(p, idx, 0, whole, err)
    ice.ice_pool4_pack(p, idx, first, part, err)
    assert ice.ice_check(err) == ice.ICE_OK
    wk, wv = (x.view(cfg.units, cfg.page_cap, S, D) for x in ref.decode(whole.view(-1, R)))
    pk, pv = (x.view(cfg.units, cfg.page_cap, S, D) for x in ref.decode(part.view(-1, R)))
    tok = idx.page_tokens
    new = (tok >= first)[..., None]
    for a, b in ((wk, pk), (wv, pv)):
        assert torch.equal(torch.where(new, a, torch.zeros_like(a)), b)


# -------------------------------------------------------------- attention --
def _one_unit(k, v, Q, dtype, scale=0.088, lens=None):
    """Attention of one KV head over pages k, v [n, 16, 128] (held in 4 bits): O, lse, and the values attended to."""
    n, hq = k.shape[0], Q.shape[0]
    p = _params(1, hq, 1, dtype)
    recs = ref.encode(k, v).view(n, 1, R)
    bt = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    O, lse, ws, err = _attn_buffers(1, hq, p)
    ln = torch.tensor([lens or n * S], dtype=torch.int32, device="cuda")
    ice.ice_cache4_attn_decode(p, Q[None].contiguous(), ice.Cache4(recs, bt), ln, scale, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    K, V = (x.reshape(-1, D)[:int(ln)] for x in ref.decode(recs[:, 0]))
    return O[0].double(), lse[0].double(), K, V


def _rms_check(O, q, K, V, scale, what=""):
    o, _ = ref.attention(q, K, V, scale)
    tol = ref.attention_rms_tolerance(q, K, V, scale)
    for h in range(q.shape[0]):
        e = float((O[h] - o[h]).norm())
        assert e <= float(tol[h]), (what, h, e / float(o[h].norm()), float(tol[h] / o[h].norm()))


HEADS = [("bf16", 4), ("bf16", 8), ("bf16", 16), ("fp32", 3), ("fp32", 8), ("fp32", 12)]


def _one_hot_check(O, lse, q, K, V, scale):
    """A head whose largest score takes all the weight (its lead is more than the scores' errors)."""
    o, l = ref.attention(q[None], K, V, scale)
    s = (q @ K.T * scale).sort(descending=True).values
    e = 16 * 2.0 ** -23 * 3 * scale * float(q.abs() @ K.abs().amax(0))
    assert float(s[0] - s[1]) > 2 * e + 60
    assert float((O - o[0]).abs().max()) <= (2.0 ** -20 + 2.0 ** -21) * float(V.abs().max())  # the weights' 22 bits
    assert abs(float(lse - l[0])) <= e


@pytest.mark.parametrize("dtype,hq", HEADS)
def test_heads_of_one_group_do_not_disturb_each_other(dtype, hq):
    """A head whose query is not finite, is large or tiny leaves the other heads of its group as they are."""
    n = 40
    k, v = (torch.randn((n, S, D), generator=_gen(s), device="cuda").bfloat16() for s in (231, 232))
    plain = torch.randn((hq, D), generator=_gen(233), device="cuda").to(DT[dtype])
    _, wlse, K, V = _one_unit(k, v, plain, dtype)
    for what in (math.inf, -math.inf, math.nan, 2.0 ** 24, 2.0 ** -60, 2.0 ** -110):
        Q = plain.clone()
        finite = math.isfinite(what)
        if finite:
            Q[1] = (Q[1].double() * what).to(DT[dtype])
        else:
            Q[1, 77] = what
        O, lse, _, _ = _one_unit(k, v, Q, dtype)
        other = [h for h in range(hq) if h != 1]
        # (not to the last bit: the group's running maxima move together)
        _rms_check(O[other], Q[other].double(), K, V, 0.088, what)
        assert float((lse[other] - wlse[other]).abs().max()) <= 2.0 ** -18, what
        if not finite:
            assert bool(O[1].isnan().all()) and bool(lse[1].isnan())
        elif what < 1:  # scores of 2^-50: the mean
            o, l = ref.attention(Q[1:2].double(), K, V, 0.088)
            to, tl = ref.attention_tolerance(Q[1:2].double(), K, V, 0.088)
            assert float((O[1] - o[0]).abs().max()) <= to and abs(float(lse[1] - l[0])) <= tl
        else:
            _one_hot_check(O[1], lse[1], Q[1].double(), K, V, 0.088)


@pytest.mark.parametrize("dtype,hq", HEADS)
def test_scores_beyond_2_to_31(dtype, hq):
    """Scores whose last place is far more than the range of exp: the largest takes it all."""
    n = 40
    k, v = (torch.randn((n, S, D), generator=_gen(s), device="cuda").bfloat16() for s in (231, 232))
    plain = torch.randn((hq, D), generator=_gen(233), device="cuda").to(DT[dtype])
    for size in (2.0 ** 34, 2.0 ** 60, 2.0 ** 100):
        for heads in (range(hq), (1,)):
            Q = plain.clone()
            for h in heads:
                Q[h] = (Q[h].double() * size).to(DT[dtype])
            O, lse, K, V = _one_unit(k, v, Q, dtype)
            for h in heads:
                _one_hot_check(O[h], lse[h], Q[h].double(), K, V, 0.088)
            other = [h for h in range(hq) if h not in heads]
            if other:
                _rms_check(O[other], Q[other].double(), K, V, 0.088, size)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_queries(dtype):
    """Queries up to the type's largest value, over keys small enough that no score overflows."""
    n, hq = 20, 4
    k, v = (torch.randn((n, S, D), generator=_gen(s), device="cuda") for s in (241, 242))
    k = (k * 2.0 ** (-115 if dtype == "bf16" else -125)).bfloat16()  # (fp32: steps are subnormal)
    Q = torch.randn((hq, D), generator=_gen(243), device="cuda")
    Q = (Q / Q.abs().max() * float(torch.finfo(torch.bfloat16).max)).to(DT[dtype])
    if dtype == "bf16":  # |scale q| stays below 2^116
        Q = (Q.double() * 2.0 ** -10).bfloat16()
    Q[2] = (Q[2].double() * 2.0 ** -100).to(DT[dtype])
    O, lse, K, V = _one_unit(k, v.bfloat16(), Q, dtype)
    for h in range(hq):
        o, l = ref.attention(Q[h:h + 1].double(), K, V, 0.088)
        to, tl = ref.attention_tolerance(Q[h:h + 1].double(), K, V, 0.088)
        assert float((O[h] - o[0]).abs().max()) <= to and abs(float(lse[h] - l[0])) <= tl, h


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [5, 100])
def test_smallest_queries_and_scales(dtype, tokens):
    """Scores far below fp32's smallest number: the mean of the values, also where a page has slots without a token."""
    n = -(-tokens // S)
    k, v = (torch.randn((n, S, D), generator=_gen(s), device="cuda").bfloat16() for s in (241, 242))
    for size, scale in ((2.0 ** -120, 1e-30), (2.0 ** -126, 1.0), (0.0, 0.088), (1.0, 1e-38), (2.0 ** -120, -1e-30)):
        Q = (torch.randn((6, D), generator=_gen(243), device="cuda") * size).to(DT[dtype])
        O, lse, K, V = _one_unit(k, v, Q, dtype, scale, tokens)
        _rms_check(O, Q.double(), K, V, scale, size)
        assert float((lse - math.log(tokens)).abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 14, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("at", [0, 3000, 4095])
@pytest.mark.parametrize("dtype,hq", [("bf16", 4), ("bf16", 8), ("bf16", 16), ("fp32", 8)])
def test_value_rows_of_no_weight(dtype, hq, at, ratio):
    """A value row that is far larger than the others, in a token without weight: the other rows keep their bits."""
    n, g = 256, _gen(251)
    base = torch.randn(D, generator=g, device="cuda")
    Q = (base + 0.5 * torch.randn((hq, D), generator=g, device="cuda")).to(DT[dtype])
    k = torch.randn((n * S, D), generator=g, device="cuda")
    v = 1 + torch.randn((n * S, D), generator=g, device="cuda")
    # scores of about -0.088 * 128 * 16 = -180: a weight of e^-180 = 2^-260 beside 2^60
    k[at], v[at] = -16 * base, v[at] * ratio
    O, lse, K, V = _one_unit(k.view(n, S, D).bfloat16(), v.view(n, S, D).bfloat16(), Q, dtype)
    _rms_check(O, Q.double(), K, V, 0.088)


@pytest.mark.parametrize("dtype,hq", [("bf16", 4), ("bf16", 8), ("bf16", 16), ("fp32", 8)])
def test_value_rows_that_only_some_heads_see(dtype, hq):
    """One token of huge values that half of the heads give all their weight, the others none."""
    n, g = 64, _gen(261)
    base = torch.randn(D, generator=g, device="cuda")
    sign = torch.where(torch.arange(hq, device="cuda") % 2 == 0, 1.0, -1.0)[:, None]
    Q = (sign * base + 0.3 * torch.randn((hq, D), generator=g, device="cuda")).to(DT[dtype])
    k = torch.randn((n * S, D), generator=g, device="cuda")
    v = 1 + torch.randn((n * S, D), generator=g, device="cuda")
    for at in (0, 500, 1023):
        k2, v2 = k.clone(), v.clone()
        k2[at], v2[at] = 16 * base, v[at] * 2.0 ** 20
        O, lse, K, V = _one_unit(k2.view(n, S, D).bfloat16(), v2.view(n, S, D).bfloat16(), Q, dtype)
        _rms_check(O, Q.double(), K, V, 0.088, at)


def test_small_values_of_large_weight():
    """A first token of small values and most of the weight beside ordinary ones, steps that rise page after page, and
    a late token that takes the weight from all before it."""
    n, g, hq = 300, _gen(271), 8
    Q = torch.randn((hq, D), generator=g, device="cuda").bfloat16()
    k = torch.randn((n * S, D), generator=g, device="cuda")
    v = 1 + torch.randn((n * S, D), generator=g, device="cuda")
    k[0], v[0] = Q.float().mean(0) * 12, v[0] * 2.0 ** -12
    rising = v * torch.exp2(torch.arange(n * S, device="cuda") / 200.0)[:, None]
    falling = v * torch.exp2(-torch.arange(n * S, device="cuda") / 200.0)[:, None]
    late = k.clone()
    late[n * S - 5] = Q.float().mean(0) * 40
    for kk, vv in ((k, v), (k, rising), (k, falling), (late, v), (late, falling), (late, rising)):
        O, lse, K, V = _one_unit(kk.view(n, S, D).bfloat16(), vv.view(n, S, D).bfloat16(), Q, "bf16")
        _rms_check(O, Q.double(), K, V, 0.088)


@pytest.mark.parametrize("dtype,hq", [("bf16", 4), ("bf16", 8), ("bf16", 16), ("fp32", 8)])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -20, 2.0 ** -7])
def test_first_token_of_all_the_weight_and_small_values(dtype, hq, size):
    """What a head attends to where it attends to nothing: the other tokens' values are far larger, their weights small."""
    n, g = 256, _gen(276)
    base = torch.randn(D, generator=g, device="cuda")
    Q = (base + 0.3 * torch.randn((hq, D), generator=g, device="cuda")).to(DT[dtype])
    k = torch.randn((n * S, D), generator=g, device="cuda")
    v = 1 + torch.randn((n * S, D), generator=g, device="cuda")
    k[0], v[0] = 2 * base, v[0] * size  # a score of about 22
    O, lse, K, V = _one_unit(k.view(n, S, D).bfloat16(), v.view(n, S, D).bfloat16(), Q, dtype)
    _rms_check(O, Q.double(), K, V, 0.088)
    k[n * S // 2], v[n * S // 2] = 2 * base, v[0]  # and once more, late
    O, lse, K, V = _one_unit(k.view(n, S, D).bfloat16(), v.view(n, S, D).bfloat16(), Q, dtype)
    _rms_check(O, Q.double(), K, V, 0.088)


@pytest.mark.parametrize("size", [1e38, 2.0 ** -100])
def test_largest_and_smallest_values(size):
    """Steps of 2^123 (three tokens: their sum stays below fp32's largest number) and of 2^-103."""
    for tokens in (1, 2, 3):
        k = torch.randn((1, S, D), generator=_gen(281), device="cuda")
        v = (torch.rand((1, S, D), generator=_gen(282), device="cuda") * 2 - 1) * size
        v[..., 0::64], v[..., 1::64] = size, -size
        Q = torch.randn((8, D), generator=_gen(283), device="cuda").bfloat16()
        O, lse, K, V = _one_unit(k.bfloat16(), v.bfloat16(), Q, "bf16", lens=tokens)
        _rms_check(O, Q.double(), K, V, 0.088)


ACCURACY = [  # hq, hkv, dtype, lens
    (4, 1, "bf16", [1, 16, 17, 300]), (32, 8, "bf16", [2049, 5]), (64, 8, "bf16", [4097]), (16, 1, "bf16", [4000, 100]),
    (4, 1, "fp32", [1, 33, 500]), (8, 1, "fp32", [1754]), (12, 1, "fp32", [900, 2]), (64, 8, "bf16", [100003]),
]


@pytest.mark.parametrize("hq,hkv,dtype,lens", ACCURACY)
def test_accuracy(hq, hkv, dtype, lens):
    """The error's norm against what independent roundings leave."""
    B, g = len(lens), hq // hkv
    p = _params(B, hq, hkv, dtype)
    blocks = -(-max(lens) // S)
    recs = _random_records(700, hkv, 291)
    bt = torch.randint(0, 700, (B, blocks), generator=_gen(292), device="cuda").int()
    Q = torch.randn((B, hq, D), generator=_gen(293), device="cuda").to(DT[dtype])
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.088,
                               O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    for b in range(B):
        for h in range(hkv):
            K, V = (x.reshape(-1, D)[:lens[b]] for x in ref.decode(recs[bt[b].long(), h]))
            hs = slice(h * g, (h + 1) * g)
            _rms_check(O[b, hs].double(), Q[b, hs].double(), K, V, 0.088, (b, h))


# ------------------------------------------------------------- many units --
def _check_units(O, lse, Q, kv_of, B, hkv, scale, only):
    g = Q.shape[1] // hkv
    for b in range(B):
        for h in range(hkv):
            hs = slice(h * g, (h + 1) * g)
            if not only(b):
                continue
            k, v = kv_of(b, h)
            q = Q[b, hs].double()
            o, l = ref.attention(q, k, v, scale)
            to, tl = ref.attention_tolerance(q, k, v, scale)
            assert float((O[b, hs].double() - o).abs().max()) <= to, (b, h)
            assert float((lse[b, hs].double() - l).abs().max()) <= tl, (b, h)


def test_more_units_than_a_cta_keeps_at_hand():
    """1280 units of ragged lengths, empty ones among them."""
    B, hq, hkv = 40, 32, 32
    g = torch.Generator().manual_seed(301)
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    lens[0], lens[7], lens[8], lens[B - 1] = 0, 0, 0, 0
    lens[20] = 1500
    p = _params(B, hq, hkv, "bf16")
    blocks = -(-max(lens) // S)
    _, bt = _cache(B, blocks, 1, 302)
    recs = _random_records(B * blocks + 2, hkv, 303)
    Q = torch.randn((B, hq, D), generator=_gen(304), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    empty = ln == 0
    assert bool((O[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())

    def kv_of(b, h):
        k, v = ref.decode(recs[bt[b, :-(-lens[b] // S)].long(), h])
        return k.reshape(-1, D)[:lens[b]], v.reshape(-1, D)[:lens[b]]

    _check_units(O, lse, Q, kv_of, B, hkv, 0.088, lambda b: lens[b] > 0)


def test_runs_that_pass_many_empty_units():
    """Long sequences with hundreds of empty ones between them: a CTA's run walks past the units it keeps at hand."""
    B, hq, hkv = 3000, 2, 1
    at = {0: 80000, 1: 33, 700: 5, 1300: 16, 1900: 160003, 2500: 1, 2501: 20, 2999: 100000}  # runs of about 70 pages
    p = _params(B, hq, hkv, "bf16")
    blocks = -(-max(at.values()) // S)
    recs = _random_records(900, hkv, 311)
    bt = torch.randint(0, 900, (B, blocks), generator=_gen(312), device="cuda").int()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for b, n in at.items():
        lens[b] = n
    Q = torch.randn((B, hq, D), generator=_gen(313), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(B, hq, p)
    for _ in range(2):
        O.fill_(7.0)
        ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), lens, 0.088, O, lse, ws, err)
        assert ice.ice_check(err) == ice.ICE_OK
        empty = lens == 0
        assert bool((O[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())

        def kv_of(b, h):
            k, v = ref.decode(recs[bt[b].long(), h])
            return k.reshape(-1, D)[:at[b]], v.reshape(-1, D)[:at[b]]

        _check_units(O, lse, Q, kv_of, B, hkv, 0.088, lambda b: b in at)


def test_selected_pages_of_many_units():
    """600 units of selected pages (none for some) and a tail that some sequences lack."""
    B, hq, hkv, P, most = 75, 16, 8, 12, 9
    U = B * hkv
    p = _params(B, hq, hkv, "bf16", page_cap=P)
    recs = _random_records(U, P, 321)
    lens = torch.randint(0, S + 1, (U, P), generator=_gen(322), device="cuda").int()
    count = torch.randint(0, most + 1, (U,), generator=_gen(323), device="cuda").int()
    sel = torch.rand((U, P), generator=_gen(324), device="cuda").argsort(1)[:, :most].int().contiguous()
    tail = torch.randint(0, 40, (B,), generator=torch.Generator().manual_seed(325)).tolist()
    tail[0] = tail[30] = 0
    count[:hkv] = 0  # sequence 0: nothing at all
    _, bt = _cache(B, 3, 1, 326)
    trec = _poison(_random_records(B * 3 + 2, hkv, 327), bt, tail, hkv)
    Q = torch.randn((B, hq, D), generator=_gen(328), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ice.ice_sparse_attn_decode4(p, Q, recs, lens, sel, count, ice.Cache4(trec, bt),
                                torch.tensor(tail, dtype=torch.int32, device="cuda"), 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    assert bool((O[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    tk, tv = _rows_of(trec, bt, 0)
    slot = torch.arange(S, device="cuda")

    def kv_of(b, h):
        u = b * hkv + h
        pg = sel[u, :int(count[u])].long()
        ok = slot < lens[u, pg][:, None]
        k, v = (x[ok] for x in ref.decode(recs[u, pg]))
        return torch.cat((k, tk[b, h, :tail[b]])), torch.cat((v, tv[b, h, :tail[b]]))

    _check_units(O, lse, Q, kv_of, B, hkv, 0.088,
                 lambda b: b > 0 and (tail[b] > 0 or int(count[b * hkv:b * hkv + hkv].min()) > 0))
