"""Norm and rotation, the 4-bit paged cache, the 4-bit pool and the attention over both, against the 64-bit
restatement in cache4_ref.py."""
import math

import pytest
import torch

import cache4_ref as ref
import semantic_paged_kv_gb300 as ice

pytestmark = pytest.mark.gpu
D, S, R = 128, 16, 2304
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step of the storage type, relative
FILL = 0xAB


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _params(B, hq, hkv, dtype, page_cap=1, **kw):
    return ice.Config(batch=B, n_q_heads=hq, n_kv_heads=hkv, n_tokens=0, np_cap=1, page_cap=page_cap,
                      dtype=ice.ICE_BF16 if dtype == "bf16" else ice.ICE_FP32, **kw).params()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _table(rd, n, base=5e5):
    inv = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    t = torch.empty((n, rd // 2, 2), dtype=torch.float32, device="cuda")
    ice.ice_rope_table(inv, n, t)
    return inv, t


def test_rope_table_far_positions():
    inv, t = _table(128, 200001)
    at = torch.tensor([0, 1, 2, 4095, 99999, 200000], device="cuda")
    a = at.double()[:, None] * inv
    want = torch.stack((a.cos(), a.sin()), -1)
    # one rounding to fp32 of values up to 1, and 1e-11 for an angle of 2e5 in fp64
    assert float((t[at].double() - want).abs().max()) <= 2.0 ** -25 + 1e-10


def _qkv(B, T, hq, hkv, dtype, seed, scale=1.0):
    x = (scale * torch.randn((B, T, hq + 2 * hkv, D), generator=_gen(seed), device="cuda")).to(DT[dtype])
    return x, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]


ROPE = [  # B, T, hq, hkv, dtype, rd, interleaved, norm
    (1, 1, 4, 1, "fp32", 128, False, False), (3, 1, 64, 8, "bf16", 128, False, True),
    (2, 37, 32, 8, "bf16", 128, True, False), (1, 129, 6, 6, "bf16", 64, False, True),
    (2, 5, 8, 2, "fp32", 96, False, True), (1, 33, 5, 5, "fp32", 16, True, True),
    (1, 2, 16, 1, "bf16", 96, True, True), (4, 3, 24, 2, "bf16", 112, False, False),
    (1, 1000, 2, 1, "bf16", 128, False, True), (2, 7, 7, 7, "bf16", 0, False, True),
]


@pytest.mark.parametrize("B,T,hq,hkv,dtype,rd,inter,norm", ROPE)
def test_qkv_rope(B, T, hq, hkv, dtype, rd, inter, norm):
    p = _params(B, hq, hkv, dtype)
    x, q, k, v = _qkv(B, T, hq, hkv, dtype, 1)
    n_pos = 70000
    table = _table(rd, n_pos)[1] if rd else None
    pos = torch.randint(0, n_pos, (B, T), generator=_gen(2), device="cuda").int()
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=_gen(s), device="cuda")).to(DT[dtype]) for s in (3, 4))
    rope = ice.Rope(table, interleaved=inter, q_norm=wq if norm else None, k_norm=wk if norm else None, eps=1e-5)
    qo = torch.full((B, T, hq, D), 7.0, dtype=DT[dtype], device="cuda")
    ko, vo = (torch.full((B, hkv, T, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    counts = torch.tensor([T - (b % 2) * (T // 2) for b in range(B)], dtype=torch.int32, device="cuda")
    err = _err()
    ice.ice_qkv_rope(p, T, ice.rows(q), ice.rows(k), ice.rows(v), pos, None, counts, rope, ice.rows(qo),
                     ice.rows(ko.transpose(1, 2)), ice.rows(vo.transpose(1, 2)), err)
    assert ice.ice_check(err) == ice.ICE_OK
    live = torch.arange(T, device="cuda") < counts[:, None]
    for inp, w, out in ((q, wq, qo), (k, wk, ko.transpose(1, 2))):
        y = ref.norm(inp, w, 1e-5) if norm else inp.double()
        size = y.abs()
        if rd:
            size = ref.rotate(size, torch.ones_like(table[pos.long()]), inter).abs() + 2 * size
            y = ref.rotate(y, table[pos.long()], inter)
        # norm: mean, eps, root and two products; rotation: two products and a sum -- at most 8 roundings in fp32
        tol = STEP[dtype] * y.abs() + 8 * 2.0 ** -24 * 2 * size.amax(-1, keepdim=True) * (1 if rd or norm else 0)
        assert bool(((out.double() - y).abs() <= tol)[live].all())
        assert bool((out == 7)[~live].all())
    assert torch.equal(vo.transpose(1, 2)[live], v[live]) and bool((vo.transpose(1, 2) == 7)[~live].all())


def test_qkv_rope_in_place_start_and_parts():
    """In place on a packed projection, positions from start, each of q, k and v alone: the same bits."""
    B, T, hq, hkv = 3, 21, 8, 2
    p = _params(B, hq, hkv, "bf16")
    x, q, k, v = _qkv(B, T, hq, hkv, "bf16", 5)
    _, table = _table(128, 5000)
    rope = ice.Rope(table, q_norm=x[0, 0, 0].clone(), k_norm=x[0, 0, 1].clone())
    start = torch.tensor([0, 7, 4979], dtype=torch.int32, device="cuda")
    pos = start[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
    want = [torch.zeros_like(t) for t in (q, k, v)]
    err = _err()
    r = ice.rows
    ice.ice_qkv_rope(p, T, r(q), r(k), r(v), pos.contiguous(), None, None, rope, *(r(t) for t in want), err)
    one = [torch.zeros_like(t) for t in (q, k, v)]
    ice.ice_qkv_rope(p, T, r(q), None, None, None, start, None, rope, r(one[0]), None, None, err)
    ice.ice_qkv_rope(p, T, None, r(k), None, None, start, None, rope, None, r(one[1]), None, err)
    ice.ice_qkv_rope(p, T, None, None, r(v), None, start, None, rope, None, None, r(one[2]), err)
    ice.ice_qkv_rope(p, T, r(q), r(k), r(v), None, start, None, rope, r(q), r(k), r(v), err)
    assert ice.ice_check(err) == ice.ICE_OK
    for a, b, c in zip(want, one, (q, k, v)):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_qkv_rope_position_outside_the_table():
    B, T, hq, hkv = 2, 3, 4, 2
    p = _params(B, hq, hkv, "bf16")
    _, q, k, v = _qkv(B, T, hq, hkv, "bf16", 6)
    _, table = _table(128, 100)
    out = [torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in (q, k, v)]
    pos = torch.tensor([[0, 100, 99], [-1, 5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    err = _err()
    ice.ice_qkv_rope(p, T, *(ice.rows(t) for t in (q, k, v)), pos, None, None, ice.Rope(table),
                     *(ice.rows(t) for t in out), err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    ok = (pos >= 0) & (pos < 100)
    for o in out:
        assert bool((o == 7)[~ok].all()) and not bool((o == 7)[ok].all(-1).any())
    # empty calls
    ice.ice_qkv_rope(p, 0, *(ice.rows(t) for t in (q, k, v)), pos, None, None, None, *(ice.rows(t) for t in out), err)
    ice.ice_qkv_rope(p, T, None, None, None, None, None, None, None, None, None, None, err)
    assert ice.ice_check(err) == ice.ICE_OK


# ------------------------------------------------------------------ cache --
def _cache(B, blocks, hkv, seed, extra=2):
    n = B * blocks + extra
    table = torch.randperm(n, generator=_gen(seed), device="cuda")[:B * blocks].view(B, blocks).int().contiguous()
    return torch.full((n, hkv, R), FILL, dtype=torch.uint8, device="cuda"), table


def _rows_of(recs, table, lens_max):
    """K, V [B, Hkv, blocks * 16, 128] in 64 bits."""
    r = recs[table.long()]
    k, v = ref.decode(r.reshape(-1, R))
    sh = (*r.shape[:3], S, D)
    return tuple(x.view(sh).transpose(1, 2).reshape(r.shape[0], r.shape[2], -1, D) for x in (k, v))


APPEND = [  # B, T, hq, hkv, dtype, rd, interleaved, norm, starts
    (1, 1, 4, 1, "fp32", 128, False, False, [0]), (3, 1, 32, 8, "bf16", 128, False, False, [0, 15, 16]),
    (2, 16, 8, 2, "bf16", 128, True, False, [0, 16]), (2, 17, 6, 3, "bf16", 96, False, False, [5, 31]),
    (3, 50, 4, 4, "fp32", 64, True, False, [1, 14, 33]), (2, 100, 16, 1, "bf16", 128, False, True, [3, 64]),
    (1, 333, 8, 8, "bf16", 0, False, False, [77]),
]


@pytest.mark.parametrize("B,T,hq,hkv,dtype,rd,inter,norm,starts", APPEND)
def test_append_and_read(B, T, hq, hkv, dtype, rd, inter, norm, starts):
    p = _params(B, hq, hkv, dtype)
    _, q, k, v = _qkv(B, T, hq, hkv, dtype, 11)
    table = _table(rd, 1000)[1] if rd else None
    w = (1 + 0.3 * torch.randn(D, generator=_gen(3), device="cuda")).to(DT[dtype])
    rope = ice.Rope(table, interleaved=inter, q_norm=w if norm else None, k_norm=w if norm else None)
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    counts = torch.tensor([T - (b % 2) * (T // 3) for b in range(B)], dtype=torch.int32, device="cuda")
    blocks = (max(starts) + T) // S + 2
    recs, bt = _cache(B, blocks, hkv, 12)
    cache = ice.Cache4(recs, bt)
    qo = torch.full((B, T, hq, D), 7.0, dtype=DT[dtype], device="cuda")
    err = _err()
    r = ice.rows
    ice.ice_cache4_append(p, T, r(q), r(k), r(v), None, start, counts, rope, r(qo), cache, err)
    assert ice.ice_check(err) == ice.ICE_OK
    # the rotated rows, as ice_qkv_rope gives them (tested above); fp32 keys in 64 bits, rounded once
    q2, k2 = torch.full_like(qo, 7.0), torch.full((B, T, hkv, D), 7.0, dtype=DT[dtype], device="cuda")
    ice.ice_qkv_rope(p, T, r(q), r(k), None, None, start, counts, rope, r(q2), r(k2), None, err)
    assert torch.equal(qo, q2)
    if dtype == "fp32":
        pos = (start[:, None] + torch.arange(T, device="cuda")).long()
        k2 = ref.rotate(k.double(), table[pos], inter).float()
    want = torch.full_like(recs, FILL)
    buf = torch.empty((B, hkv, blocks * S, D), dtype=DT[dtype], device="cuda").normal_(generator=_gen(1))
    kv = [buf.clone(), buf.clone()]
    new = torch.zeros((B, blocks * S), dtype=torch.bool, device="cuda")
    for b in range(B):
        a, n = starts[b], int(counts[b])
        kv[0][b, :, a:a + n], kv[1][b, :, a:a + n] = k2[b, :n].transpose(0, 1), v[b, :n].transpose(0, 1)
        new[b, a:a + n] = True
    rec = ref.encode(*(x.view(B, hkv, blocks, S, D).transpose(1, 2).reshape(-1, S, D) for x in kv))
    rec = rec.view(B, blocks, hkv, R)
    mask = torch.zeros((B, blocks, R), dtype=torch.bool, device="cuda")
    at_k, at_v = ref.places("cuda")
    nb = new.view(B, blocks, S)
    for t in range(S):
        for cols in (at_k[t], at_v[t], torch.arange(1024 + 8 * t, 1032 + 8 * t), torch.arange(2176 + 8 * t, 2184 + 8 * t)):
            mask[:, :, cols.to("cuda")] |= nb[:, :, t:t + 1]
    cur = want[bt.long()]
    want[bt.long()] = torch.where(mask[:, :, None], rec, cur)
    assert torch.equal(recs, want)  # every new token's bytes, and nothing else
    # read back
    ko, vo = (torch.full((B, hkv, T, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    ice.ice_cache4_read(p, T, cache, start, counts, r(ko.transpose(1, 2)), r(vo.transpose(1, 2)), err)
    assert ice.ice_check(err) == ice.ICE_OK
    k64, v64 = _rows_of(recs, bt, 0)
    for b in range(B):
        a, n = starts[b], int(counts[b])
        for o, y in ((ko, k64), (vo, v64)):
            assert torch.equal(o[b, :, :n], y[b, :, a:a + n].float().to(DT[dtype])) and bool((o[b, :, n:] == 7).all())


@pytest.mark.parametrize("dtype,norm", [("bf16", False), ("bf16", True), ("fp32", False)])
def test_append_many_blocks(dtype, norm):
    """A call of many blocks (a warp each) writes the bytes that calls of few tokens (a warp per four slots) write, and
    the same queries."""
    B, T, hq, hkv, part = 6, 1291, 8, 8, 101  # 6 * 8 * 82 = 3936 blocks: more than 16 an SM
    p = _params(B, hq, hkv, dtype)
    _, q, k, v = _qkv(B, T, hq, hkv, dtype, 61)
    w = (1 + 0.3 * torch.randn(D, generator=_gen(3), device="cuda")).to(DT[dtype])
    rope = ice.Rope(_table(128, 1400)[1], q_norm=w if norm else None, k_norm=w if norm else None)
    start = torch.tensor([0, 15, 1, 16, 7, 90], dtype=torch.int32, device="cuda")
    counts = torch.tensor([T, T - 300, 0, 5, T, T - 1], dtype=torch.int32, device="cuda")
    recs, bt = _cache(B, (90 + T) // S + 2, hkv, 62)
    recs2, err, r = recs.clone(), _err(), ice.rows
    qo, qo2 = (torch.full((B, T, hq, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    ice.ice_cache4_append(p, T, r(q), r(k), r(v), None, start, counts, rope, r(qo), ice.Cache4(recs, bt), err)
    for a in range(0, T, part):
        n = min(part, T - a)
        x = [t[:, a:a + n] for t in (q, k, v, qo2)]
        ice.ice_cache4_append(p, n, *map(r, x[:3]), None, start + a, (counts - a).clamp(0, n), rope, r(x[3]),
                              ice.Cache4(recs2, bt), err)
    assert ice.ice_check(err) == ice.ICE_OK
    assert torch.equal(recs, recs2) and torch.equal(qo, qo2)


def test_append_refuses_on_the_device():
    """Cache positions, pages and rotation positions outside their ranges: those tokens are left out."""
    B, T, hq, hkv = 3, 20, 4, 2
    p = _params(B, hq, hkv, "bf16")
    _, q, k, v = _qkv(B, T, hq, hkv, "bf16", 21)
    recs, bt = _cache(B, 2, hkv, 22)
    bt[1, 0], bt[2, 1] = -1, recs.shape[0]
    cache, err = ice.Cache4(recs, bt), _err()
    start = torch.tensor([-3, 0, 14], dtype=torch.int32, device="cuda")
    r = ice.rows
    ice.ice_cache4_append(p, T, None, r(k), r(v), None, start, None, None, None, cache, err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    written = (recs != FILL).any(-1).any(-1)
    ok = [bt[0, 0], bt[0, 1], bt[1, 1], bt[2, 0]]  # tokens 0 .. 16 of sequence 0, 16 .. 19 of 1, 14, 15 of 2
    assert sorted(int(i) for i in ok) == sorted(written.nonzero().flatten().tolist())
    k64, _ = _rows_of(recs, torch.stack([torch.stack((bt[0, 0], bt[0, 1]))]), 0)
    want = ref.held(k[0, 3:20].transpose(0, 1))
    assert torch.equal(k64[0, :, :17], want)
    # read: the same tokens
    ko, vo = (torch.full((B, T, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ice.ice_cache4_read(p, T, cache, start, None, r(ko), r(vo), err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    left = (ko == 7).all(-1).all(-1).cpu()
    want = torch.ones((B, T), dtype=torch.bool)
    want[0, 3:], want[1, 16:], want[2, :2] = False, False, False
    assert torch.equal(left, want)
    # rotation positions
    recs.fill_(FILL)
    _, table = _table(128, 10)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    bt2 = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2).contiguous()
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    ice.ice_cache4_append(p, T, None, r(k), r(v), pos, zero, None, ice.Rope(table), None, ice.Cache4(recs, bt2), err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    meta = recs[:6].view(3, 2, hkv, R)[..., 1024:1152].reshape(3, 2, hkv, S, 8)
    wrote = (meta != FILL).any(-1).any(2).reshape(3, 32)
    assert bool(wrote[:, :10].all()) and not bool(wrote[:, 10:].any())


# ------------------------------------------------------------------- pool --
def _pool(U, P, dtype, seed):
    k = torch.randn((U, P, S, D), generator=_gen(seed), device="cuda")
    v = torch.randn((U, P, S, D), generator=_gen(seed + 1), device="cuda") * 3 + 1
    lens = torch.randint(1, S + 1, (U, P), generator=_gen(seed + 2), device="cuda").int()
    return k.to(DT[dtype]), v.to(DT[dtype]), lens


def _ix(**f):
    return ice.IceIndex(**{n: t.data_ptr() for n, t in f.items()})


@pytest.mark.parametrize("U,P,dtype", [(1, 1, "bf16"), (3, 7, "bf16"), (2, 33, "fp32"), (5, 130, "bf16")])
def test_pool_pack_and_unpack(U, P, dtype):
    p = _params(1, U, U, dtype, page_cap=P)
    k, v, lens = _pool(U, P, dtype, 31)
    lens[:, 0] = 16
    if P > 4:
        lens[0, 1] = 0
        # groups that are constant, tiny, far from zero, or not finite
        k[0, 2, 0] = 3.25
        k[0, 2, 1, :64] *= 1e-36
        k[0, 2, 2] = k[0, 2, 2] * 0.01 + 1000
        k[0, 2, 3, 70], v[0, 2, 3, 1], v[0, 2, 4, 100] = math.nan, math.inf, -math.inf
        v[0, 2, 5], v[0, 2, 6, 64:] = 0, 1e-40
        k[0, 2, 7, 0], k[0, 2, 7, 1] = 3e38, -3e38
        lens[0, 2] = 16
    n_pages = torch.tensor([P - (u % 2) for u in range(U)], dtype=torch.int32, device="cuda")
    n_pages[0] = P
    assert ice.ice_pool4_bytes(p) == U * P * R
    recs = torch.full((U, P, R), FILL, dtype=torch.uint8, device="cuda")
    err = _err()
    ice.ice_pool4_pack(p, _ix(n_pages=n_pages, page_len=lens, pool_k=k, pool_v=v), 0, recs, err)
    want = ref.encode(k.view(-1, S, D), v.view(-1, S, D)).view(U, P, R)
    used = (torch.arange(S, device="cuda") < lens[..., None])
    mask = torch.zeros((U, P, R), dtype=torch.bool, device="cuda")
    at_k, at_v = ref.places("cuda")
    for t in range(S):
        for cols in (at_k[t], at_v[t], torch.arange(1024 + 8 * t, 1032 + 8 * t), torch.arange(2176 + 8 * t, 2184 + 8 * t)):
            mask[:, :, cols.to("cuda")] |= used[:, :, t:t + 1]
    want = torch.where(mask, want, torch.zeros_like(want))
    live = torch.arange(P, device="cuda") < n_pages[:, None]
    # NaN (mid of a group that is not finite) has one bit pattern on each side
    nan = lambda r: r.view(torch.bfloat16).isnan()  # noqa: E731
    meta = torch.zeros(R // 2, dtype=torch.bool, device="cuda")
    meta[512:576], meta[1088:1152] = True, True
    a, b = recs.view(torch.int16), want.view(torch.int16)
    same = (a == b) | (nan(recs) & nan(want) & meta)
    assert bool(same[live].all()) and bool((recs == FILL)[~live].all())
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ice.ice_pool4_unpack(p, _ix(n_pages=n_pages, page_len=lens, pool_k=ko, pool_v=vo), recs, err)
    assert ice.ice_check(err) == ice.ICE_OK
    for o, x in ((ko, k), (vo, v)):
        y = torch.where(used[..., None], ref.held(x), torch.zeros_like(x, dtype=torch.float64)).float().to(DT[dtype])
        assert torch.allclose(o[live].double(), y[live].double(), rtol=0, atol=0, equal_nan=True)
        assert bool((o == 7)[~live].all())
    if P > 4:
        assert bool(ko[0, 2, 3, 64:].isnan().all()) and not bool(ko[0, 2, 3, :64].isnan().any())
        assert bool(vo[0, 2, 3, :64].isnan().all()) and bool(vo[0, 2, 4, 64:].isnan().all())
        assert bool((ko[0, 2, 0] == 3.25).all()) and bool((vo[0, 2, 5] == 0).all())


# -------------------------------------------------------------- attention --
def _random_records(n, hkv, seed, spread=1.0):
    k = torch.randn((n * hkv, S, D), generator=_gen(seed), device="cuda") * spread
    v = torch.randn((n * hkv, S, D), generator=_gen(seed + 1), device="cuda") * spread
    return ref.encode(k.bfloat16(), v.bfloat16()).view(n, hkv, R)


def _attn_buffers(B, hq, p):
    O = torch.full((B, hq, D), 7.0, device="cuda")
    lse = torch.full((B, hq), 7.0, device="cuda")
    return O, lse, ice.workspace(ice.ice_attn4_workspace_bytes(p)), _err()


def _check_attn(O, lse, Q, kv_of, B, hkv, scale):
    g = Q.shape[1] // hkv
    for b in range(B):
        for h in range(hkv):
            k, v = kv_of(b, h)
            q = Q[b, h * g:(h + 1) * g].double()
            o, l = ref.attention(q, k, v, scale)
            to, tl = ref.attention_tolerance(q, k, v, scale)
            hs = slice(h * g, (h + 1) * g)
            assert float((O[b, hs].double() - o).abs().max()) <= to, (b, h, k.shape[0])
            if lse is not None:
                if k.shape[0]:
                    assert float((lse[b, hs].double() - l).abs().max()) <= tl
                else:
                    assert bool((lse[b, hs] == -math.inf).all())


def _poison(recs, table, lens, hkv):
    """Slots behind the last token of every sequence, and pages that no sequence has, hold NaN."""
    used = torch.zeros((recs.shape[0], S), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for x in range(-(-n // S)):
            used[int(table[b, x]), :min(S, n - x * S)] = True
    for off in (1024, 2176):
        m = recs[:, :, off:off + 128].view(recs.shape[0], hkv, S, 8)
        m[~used[:, None].expand(-1, hkv, -1)] = 0xFF
    return recs


ATTN = [  # hq, hkv, dtype, lens
    (4, 1, "fp32", [1, 0, 16, 17]), (4, 1, "bf16", [1, 15, 16, 17, 0, 33]), (32, 8, "bf16", [1000]),
    (32, 32, "bf16", [100, 257]), (64, 8, "bf16", [5, 640, 0, 129]), (16, 1, "bf16", [3000, 1]),
    (9, 1, "bf16", [77]), (13, 1, "fp32", [130, 2]), (24, 2, "bf16", [555, 48]), (10, 5, "fp32", [100, 31]),
    (8, 8, "fp32", [4097]), (6, 2, "bf16", [0, 0]), (40, 8, "bf16", [65, 64, 63]),
]


@pytest.mark.parametrize("hq,hkv,dtype,lens", ATTN)
def test_cache_attention(hq, hkv, dtype, lens):
    B = len(lens)
    p = _params(B, hq, hkv, dtype)
    blocks = max(1, -(-max(lens) // S)) + 1
    _, bt = _cache(B, blocks, 1, 41)
    recs = _poison(_random_records(B * blocks + 2, hkv, 42), bt, lens, hkv)
    Q = torch.randn((B, hq, D), generator=_gen(43), device="cuda").to(DT[dtype])
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    k, v = _rows_of(recs, bt, 0)
    _check_attn(O, lse, Q, lambda b, h: (k[b, h, :lens[b]], v[b, h, :lens[b]]), B, hkv, 0.088)
    # again with the same workspace and no lse: the same bits
    O2 = torch.full_like(O, 3.0)
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, 0.088, O2, None, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK and torch.equal(O, O2)


@pytest.mark.parametrize("hq,hkv,dtype,tail", [(4, 1, "fp32", [5, 0]), (64, 8, "bf16", [0, 33, 16]),
                                               (32, 8, "bf16", None), (16, 1, "bf16", [100]), (32, 32, "bf16", [1])])
def test_sparse_attention(hq, hkv, dtype, tail):
    B = len(tail) if tail else 2
    U, P, most = B * hkv, 50, 20
    p = _params(B, hq, hkv, dtype, page_cap=P)
    recs = _random_records(U, P, 51)
    lens = torch.randint(1, S + 1, (U, P), generator=_gen(52), device="cuda").int()
    lens[0, :3] = 0
    pad = torch.arange(S, device="cuda") >= lens[..., None]
    for off in (1024, 2176):
        recs[:, :, off:off + 128].view(U, P, S, 8)[pad] = 0xFF
    count = torch.randint(0, most + 1, (U,), generator=_gen(53), device="cuda").int()
    count[0] = 3
    if U > 1:
        count[1] = 0
    sel = torch.rand((U, P), generator=_gen(54), device="cuda").argsort(1)[:, :most].int().contiguous()
    sel[0, :3] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")  # pages of no token
    Q = torch.randn((B, hq, D), generator=_gen(55), device="cuda").to(DT[dtype])
    O, lse, ws, err = _attn_buffers(B, hq, p)
    cache = ln = None
    if tail:
        blocks = max(1, -(-max(tail) // S))
        _, bt = _cache(B, blocks, 1, 56)
        trec = _poison(_random_records(B * blocks + 2, hkv, 57), bt, tail, hkv)
        cache, ln = ice.Cache4(trec, bt), torch.tensor(tail, dtype=torch.int32, device="cuda")
        tk, tv = _rows_of(trec, bt, 0)
    ice.ice_sparse_attn_decode4(p, Q, recs, lens, sel, count, cache, ln, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK

    def kv_of(b, h):
        u = b * hkv + h
        at = sel[u, :int(count[u])].long()
        ok = ~pad[u, at]
        k, v = (x[ok] for x in ref.decode(recs[u, at]))
        if tail:
            k, v = torch.cat((k, tk[b, h, :tail[b]])), torch.cat((v, tv[b, h, :tail[b]]))
        return k, v

    _check_attn(O, lse, Q, kv_of, B, hkv, 0.088)


def test_attention_large_scores_and_uneven_values():
    """Scores far apart, one token that takes the weight late, value rows of very different size."""
    p = _params(1, 8, 1, "bf16")
    n = 700
    k = torch.randn((44, S, D), generator=_gen(61), device="cuda") * 4
    v = torch.randn((44, S, D), generator=_gen(62), device="cuda")
    v *= torch.exp2(torch.randint(-20, 6, (44, S, 1), generator=_gen(63), device="cuda").float())
    Q = (torch.randn((1, 8, D), generator=_gen(64), device="cuda") * 3).bfloat16()
    k[43, 11] = Q[0, 3].float() * 2
    recs = ref.encode(k.bfloat16(), v.bfloat16()).view(44, 1, R)
    bt = torch.arange(44, dtype=torch.int32, device="cuda").view(1, 44)
    O, lse, ws, err = _attn_buffers(1, 8, p)
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), torch.tensor([n], dtype=torch.int32, device="cuda"), 0.088,
                               O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    K, V = _rows_of(recs, bt, 0)
    _check_attn(O, lse, Q, lambda b, h: (K[b, h, :n], V[b, h, :n]), 1, 1, 0.088)


def test_attention_bad_pages_and_lengths():
    hq, hkv, B = 8, 2, 3
    p = _params(B, hq, hkv, "bf16")
    _, bt = _cache(B, 4, 1, 71)
    recs = _random_records(14, hkv, 72)
    lens = [60, 64, 64]
    K, V = _rows_of(recs, bt, 0)
    ln = torch.tensor([60, 1000, -5], dtype=torch.int32, device="cuda")  # beyond the table; negative
    bt2 = bt.clone()
    bt2[0, 1], bt2[1, 3] = 14, -7
    Q = torch.randn((B, hq, D), generator=_gen(73), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt2), ln, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    keep = [[0, 2, 3], [0, 1, 2], []]

    def kv_of(b, h):
        at = [t for x in keep[b] for t in range(x * S, min(x * S + S, lens[b]))]
        return K[b, h, at], V[b, h, at]

    _check_attn(O, lse, Q, kv_of, B, hkv, 0.088)
    # selected pages outside the pool
    pool = _random_records(B * hkv, 5, 74)
    pl = torch.full((B * hkv, 5), 16, dtype=torch.int32, device="cuda")
    sel = torch.tensor([[0, 5, -1, 4]] * (B * hkv), dtype=torch.int32, device="cuda")
    cnt = torch.full((B * hkv,), 9, dtype=torch.int32, device="cuda")  # clamped to 4
    p5 = _params(B, hq, hkv, "bf16", page_cap=5)
    ice.ice_sparse_attn_decode4(p5, Q, pool, pl, sel, cnt, None, None, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY
    _check_attn(O, lse, Q, lambda b, h: tuple(x.reshape(-1, D) for x in ref.decode(pool[b * hkv + h, [0, 4]])), B, hkv,
                0.088)


def test_attention_captured_graph_and_other_stream():
    """A step (append, attend) captured once and replayed as the sequences grow; another stream than the default."""
    B, hq, hkv, steps = 2, 8, 2, 40
    p = _params(B, hq, hkv, "bf16")
    recs, bt = _cache(B, 4, hkv, 81)
    cache = ice.Cache4(recs, bt)
    x, q, k, v = _qkv(B, 1, hq, hkv, "bf16", 82)
    _, table = _table(128, 64)
    rope = ice.Rope(table)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    qo = torch.zeros((B, 1, hq, D), dtype=torch.bfloat16, device="cuda")
    O, lse, ws, err = _attn_buffers(B, hq, p)
    side = torch.cuda.Stream()

    def step():
        ice.ice_cache4_append(p, 1, ice.rows(q), ice.rows(k), ice.rows(v), None, start, None, rope, ice.rows(qo),
                              cache, err)
        lens.add_(1)
        ice.ice_cache4_attn_decode(p, qo, cache, lens, 0.088, O, lse, ws, err)
        start.add_(1)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    recs.fill_(FILL)
    start.zero_()
    lens.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(steps):
        x.copy_(torch.randn(x.shape, generator=_gen(900 + i), device="cuda"))
        g.replay()
        if i in (0, 1, 15, 16, steps - 1):
            assert ice.ice_check(err) == ice.ICE_OK
            K, V = _rows_of(recs, bt, 0)
            _check_attn(O, lse, qo[:, 0], lambda b, h: (K[b, h, :i + 1], V[b, h, :i + 1]), B, hkv, 0.088)


# ------------------------------------------------------------ used together --
def test_prompt_then_steps_over_a_4bit_pool_and_tail():
    """A prompt's projection -> rotation -> index -> 4-bit pool, its bf16 pool given back; then steps whose new tokens
    go to a 4-bit cache and whose attention covers the selected pages and that cache in one softmax."""
    B, hq, hkv, N, T, budget, steps = 2, 8, 2, 700, 700, 64, 20
    cfg = ice.Config(batch=B, n_q_heads=hq, n_kv_heads=hkv, n_tokens=N, seed=3)
    p = cfg.params()
    _, q, k, v = _qkv(B, T, hq, hkv, "bf16", 91)
    _, table = _table(128, N + steps)
    w = (1 + 0.2 * torch.randn(D, generator=_gen(92), device="cuda")).bfloat16()
    rope, err, r = ice.Rope(table, q_norm=w, k_norm=w), _err(), ice.rows
    K, V = (torch.empty((B, hkv, N, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ice.ice_qkv_rope(p, T, None, r(k), r(v), None, None, None, rope, None, r(K.transpose(1, 2)), r(V.transpose(1, 2)),
                     err)
    idx = ice.Index(cfg)
    ice.ice_build_index(p, K, V, idx, ice.workspace(ice.ice_build_workspace_bytes(p)), err)
    recs = torch.zeros(ice.ice_pool4_bytes(p), dtype=torch.uint8, device="cuda").view(cfg.units, cfg.page_cap, R)
    ice.ice_pool4_pack(p, idx, 0, recs, err)
    assert ice.ice_check(err) == ice.ICE_OK
    bare = ice.IceIndex.from_buffer_copy(idx.struct)
    bare.pool_k = bare.pool_v = None  # the selection needs none of the pool
    trec, bt = _cache(B, -(-steps // S), hkv, 93)
    tail = ice.Cache4(trec, bt)
    buf = ice.DecodeBuffers(cfg, budget)
    O, lse, ws, err = _attn_buffers(B, hq, p)
    kp = (idx.page_len, recs)
    for i in range(steps):
        _, q1, k1, v1 = _qkv(B, 1, hq, hkv, "bf16", 100 + i)
        at = torch.full((B,), i, dtype=torch.int32, device="cuda")
        pos = torch.full((B, 1), N + i, dtype=torch.int32, device="cuda")
        qo = torch.empty((B, 1, hq, D), dtype=torch.bfloat16, device="cuda")
        ice.ice_cache4_append(p, 1, r(q1), r(k1), r(v1), pos, at, None, rope, r(qo), tail, err)
        ice.ice_select_pages(p, bare, qo, budget, buf.sel_pages, buf.sel_count, buf.ws, err)
        ice.ice_sparse_attn_decode4(p, qo, recs, kp[0], buf.sel_pages, buf.sel_count, tail, at + 1, 0.088, O, lse, ws,
                                    err)
        assert ice.ice_check(err) == ice.ICE_OK
        tk, tv = _rows_of(trec, bt, 0)

        def kv_of(b, h):
            u = b * hkv + h
            pg = buf.sel_pages[u, :int(buf.sel_count[u])].long()
            tok = idx.page_tokens[u, pg]
            tok = tok[tok >= 0].long()
            # the prompt's own rows, held in 4 bits
            return (torch.cat((ref.held(K[b, h, tok]), tk[b, h, :i + 1])),
                    torch.cat((ref.held(V[b, h, tok]), tv[b, h, :i + 1])))

        _check_attn(O, lse, qo[:, 0], kv_of, B, hkv, 0.088)


def test_pack_of_inserted_tokens():
    """ice_insert_tokens, then ice_pool4_pack of the new tokens only: the pool's records are those of a whole pack."""
    B, hq, hkv, N, steps = 2, 4, 2, 300, 40
    cfg = ice.Config(batch=B, n_q_heads=hq, n_kv_heads=hkv, n_tokens=N, n_cap=N + steps, seed=5)
    p = cfg.params()
    K, V = (torch.randn((B, hkv, N, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    idx, err = ice.Index(cfg), _err()
    ice.ice_build_index(p, K, V, idx, ice.workspace(ice.ice_build_workspace_bytes(p)), err)
    recs = torch.zeros(ice.ice_pool4_bytes(p), dtype=torch.uint8, device="cuda").view(cfg.units, cfg.page_cap, R)
    ice.ice_pool4_pack(p, idx, 0, recs, err)
    iws = ice.workspace(ice.ice_insert_workspace_bytes(p))
    for i in range(steps):
        kn, vn = (torch.randn((B, hkv, D), generator=_gen(1000 + 2 * i + s), device="cuda").bfloat16() for s in (0, 1))
        ice.ice_insert_tokens(p, idx, kn, vn, iws, err)
        if i % 3 == 2 or i == steps - 1:  # one to three tokens at a time
            ice.ice_pool4_pack(p, idx, N + i // 3 * 3, recs, err)
    assert ice.ice_check(err) == ice.ICE_OK
    whole = torch.zeros_like(recs)
    ice.ice_pool4_pack(p, idx, 0, whole, err)
    assert ice.ice_check(err) == ice.ICE_OK and torch.equal(recs, whole)
    # a token whose page lies outside the capacity
    idx.token_page[0, N + steps - 1] = cfg.page_cap
    before = recs.clone()
    ice.ice_pool4_pack(p, idx, N + steps - 1, recs, err)
    assert ice.ice_check(err) == ice.ICE_ERR_CAPACITY and torch.equal(recs, before)


# --------------------------------------------------------- what tests miss --
def test_codes_on_borders():
    """Values on a coarse grid: true ties between two codes, mid a multiple of step or next to one, tiny values beside
    large ones."""
    g = _gen(111)
    n = 4000

    def ints(lo, hi):
        return torch.randint(lo, hi, (n, S, D), generator=g, device="cuda").float()

    rows = [ints(-15, 16), ints(0, 16) * 0.5, ints(-128, 128) / 16, ints(-7, 8) * 0.75 + 1.5,
            ints(-30, 31) * torch.exp2(torch.randint(-12, 3, (n, S, D), generator=g, device="cuda").float()),
            ints(-3, 4) * 1e-30, (ints(0, 31) + 100) * 2]
    rows[0][:, :, ::7] *= 1e-6
    for x in rows:
        k = x.bfloat16()
        v = k.flip(-1)
        pool = lambda t: t.view(1, n, S, D).contiguous()  # noqa: E731
        lens = torch.full((1, n), 16, dtype=torch.int32, device="cuda")
        cnt = torch.full((1,), n, dtype=torch.int32, device="cuda")
        recs, err = torch.empty((1, n, R), dtype=torch.uint8, device="cuda"), _err()
        ice.ice_pool4_pack(_params(1, 1, 1, "bf16", page_cap=n), _ix(n_pages=cnt, page_len=lens, pool_k=pool(k),
                                                                      pool_v=pool(v)), 0, recs, err)
        assert ice.ice_check(err) == ice.ICE_OK and torch.equal(recs[0], ref.encode(k, v))


def test_fp32_codes_next_to_borders():
    """fp32 values on the borders between two codes and up to some units in the last place beside them."""
    n, g = 3000, _gen(131)
    x = torch.randn((n, S, 2, D // 2), generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-40, 40, (n, S, 2, 1), generator=g, device="cuda").float())
    x += torch.randint(-2, 3, (n, S, 2, 1), generator=g, device="cuda") * x.abs().amax(-1, keepdim=True)
    meta, _ = ref.groups(x.reshape(n, S, D))
    step, mid = (meta.view(n, S, 2, 2)[..., i:i + 1].double() for i in range(2))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    at = torch.randint(-7, 8, x.shape, generator=g, device="cuda")
    near = (mid + at * step).float()
    ulps = torch.randint(-9, 10, x.shape, generator=g, device="cuda")
    near = (near.double() + ulps * torch.where(near == 0, 1e-30, near.abs().double() * 2.0 ** -24)).float()
    near = torch.minimum(torch.maximum(near, lo), hi)
    keep = (x == lo) | (x == hi) | (torch.arange(n, device="cuda") % 3 == 0)[:, None, None, None]
    k = torch.where(keep, x, near).reshape(n, S, D)
    assert torch.equal(ref.groups(k)[0], meta)  # the extremes are as they were
    v = k.flip(0).contiguous()
    lens = torch.full((1, n), S, dtype=torch.int32, device="cuda")
    cnt = torch.full((1,), n, dtype=torch.int32, device="cuda")
    recs, err = torch.empty((1, n, R), dtype=torch.uint8, device="cuda"), _err()
    ice.ice_pool4_pack(_params(1, 1, 1, "fp32", page_cap=n), _ix(n_pages=cnt, page_len=lens, pool_k=k, pool_v=v), 0,
                       recs, err)
    assert ice.ice_check(err) == ice.ICE_OK and torch.equal(recs[0], ref.encode(k, v))


def test_long_context_of_shared_pages():
    """100k tokens a sequence (the warps' sums are flushed on the way), sequences sharing the pages of a small cache."""
    B, hq, hkv, n = 2, 64, 8, 100003
    p = _params(B, hq, hkv, "bf16")
    recs = _random_records(600, hkv, 121)
    bt = torch.randint(0, 600, (B, -(-n // S)), generator=_gen(122), device="cuda").int()
    Q = torch.randn((B, hq, D), generator=_gen(123), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ln = torch.tensor([n, n - 40000], dtype=torch.int32, device="cuda")
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    for b, h in ((0, 0), (0, 7), (1, 3)):
        k, v = (x.reshape(-1, D)[:int(ln[b])] for x in ref.decode(recs[bt[b].long(), h]))
        o, l = ref.attention(Q[b, 8 * h:8 * h + 8].double(), k, v, 0.088)
        got = O[b, 8 * h:8 * h + 8].double()
        # a mean over 1e5 values: relative to its own size, as fp32 sums of that many terms leave it
        assert float((got - o).norm() / o.norm()) < 1e-5
        assert float((lse[b, 8 * h:8 * h + 8].double() - l).abs().max()) < 1e-5


def test_records_beyond_4_gb():
    """Pages whose bytes start behind 2^32."""
    n, B, hq, hkv, T = 1_900_000, 1, 4, 1, 40
    p = _params(B, hq, hkv, "bf16")
    recs = torch.zeros((n, hkv, R), dtype=torch.uint8, device="cuda")
    bt = torch.tensor([[n - 1, 5, n - 2]], dtype=torch.int32, device="cuda")
    cache, err, r = ice.Cache4(recs, bt), _err(), ice.rows
    _, q, k, v = _qkv(B, T, hq, hkv, "bf16", 131)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    ice.ice_cache4_append(p, T, None, r(k), r(v), None, start, None, None, None, cache, err)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    ice.ice_cache4_read(p, T, cache, start, None, r(ko), r(vo), err)
    O, lse, ws, err = _attn_buffers(B, hq, p)
    Q = q[:, 0].contiguous()
    ice.ice_cache4_attn_decode(p, Q, cache, start + T, 0.088, O, lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    hk, hv = ref.held(k[0, :, 0]), ref.held(v[0, :, 0])
    assert torch.equal(ko[0, :, 0], hk.bfloat16()) and torch.equal(vo[0, :, 0], hv.bfloat16())
    _check_attn(O, lse, Q, lambda b, h: (hk, hv), B, hkv, 0.088)
    # the same records as a pool: unit 0 of one, page n - 1 selected
    pl = torch.full((1, n), 16, dtype=torch.int32, device="cuda")
    sel = torch.tensor([[5, n - 1]], dtype=torch.int32, device="cuda")
    cnt = torch.full((1,), 2, dtype=torch.int32, device="cuda")
    ice.ice_sparse_attn_decode4(_params(B, hq, hkv, "bf16", page_cap=n), Q, recs, pl, sel, cnt, None, None, 0.088, O,
                                lse, ws, err)
    assert ice.ice_check(err) == ice.ICE_OK
    order = list(range(16, 32)) + list(range(16))
    _check_attn(O, lse, Q, lambda b, h: (hk[order], hv[order]), B, hkv, 0.088)


def test_one_workspace_for_several_shapes_and_two_streams():
    """One workspace for calls of different shapes, one after the other; two calls at once, a workspace each."""
    shapes = [(1, 8, 8, [3000]), (40, 32, 8, [70] * 40), (1, 16, 1, [2000]), (3, 4, 1, [500, 0, 33])]
    calls = []
    for i, (B, hq, hkv, lens) in enumerate(shapes):
        blocks = -(-max(lens) // S)
        recs = _random_records(B * blocks, hkv, 141 + i)
        bt = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
        Q = torch.randn((B, hq, D), generator=_gen(150 + i), device="cuda").bfloat16()
        calls.append((_params(B, hq, hkv, "bf16"), Q, ice.Cache4(recs, bt),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), B, hq))
    ws = ice.workspace(max(ice.ice_attn4_workspace_bytes(c[0]) for c in calls))
    err, want = _err(), []

    def call(c, w, stream=None):
        O = torch.empty((c[4], c[5], D), device="cuda")
        ice.ice_cache4_attn_decode(c[0], c[1], c[2], c[3], 0.088, O, None, w, err, stream)
        return O

    for c in calls:
        want.append(call(c, ice.workspace(ice.ice_attn4_workspace_bytes(c[0]))))
    for _ in range(3):
        for c, x in zip(calls, want):
            assert torch.equal(call(c, ws), x)
    streams = [torch.cuda.Stream() for _ in range(2)]
    own = [ice.workspace(ws.numel()) for _ in streams]
    torch.cuda.synchronize()
    got = [[call(calls[(i + j) % 4], own[j], s) for j, s in enumerate(streams)] for i in range(8)]
    torch.cuda.synchronize()
    for i in range(8):
        for j in range(2):
            assert torch.equal(got[i][j], want[(i + j) % 4])
    assert ice.ice_check(err) == ice.ICE_OK


def test_host_pool_in_4_bits():
    """A pool in pinned host memory packed from there: the records of the same pool in device memory."""
    kw = dict(batch=1, n_q_heads=8, n_kv_heads=2, n_tokens=600, seed=9)
    K, V = (torch.randn((1, 2, 600, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    cfg = ice.Config(**kw)
    p, got, err = cfg.params(), [], _err()
    hp = ice.HostPool(cfg, 64, n_threads=2)
    try:
        for pool in (None, hp):
            idx = ice.Index(cfg, host_pool=pool)
            ice.ice_build_index(p, K, V, idx, ice.workspace(ice.ice_build_workspace_bytes(p)), err)
            recs = torch.zeros((2, cfg.page_cap, R), dtype=torch.uint8, device="cuda")
            ice.ice_pool4_pack(p, idx, 0, recs, err)
            assert ice.ice_check(err) == ice.ICE_OK
            got.append((idx.n_pages.clone(), recs))
    finally:
        hp.close()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_host_pool_staging_starts_at_zero():
    """Slots that no page has filled are zero, also in memory that another pool has used before."""
    cfg = ice.Config(batch=1, n_q_heads=8, n_kv_heads=2, n_tokens=600)
    U, n = cfg.units, 64
    assert cfg.page_cap >= n
    sel = torch.arange(n, dtype=torch.int32).expand(U, n).contiguous()
    lens = torch.full((U, cfg.page_cap), S, dtype=torch.int32)
    for count in (n, 1, 0):
        hp = ice.HostPool(cfg, n, n_threads=2)
        try:
            dst = torch.full((hp.staging_bytes,), FILL, dtype=torch.uint8, device="cuda")
            for which in "kv":
                hp.host_array(which)[:] = 0x3F80
            cnt = torch.full((U,), count, dtype=torch.int32)
            ice.ice_host_pool_gather_h2d(hp, cfg.params(), sel, cnt, lens, n, dst)
            torch.cuda.synchronize()
        finally:
            hp.close()
        kv = dst[:2 * U * n * S * D * 2].view(2, U, n, -1)
        assert int(kv[:, :, count:].count_nonzero()) == 0 and bool(kv[:, :, :count].any(-1).all())


MANY_RUNS = [  # hq, hkv, dtype, lens: units whose partial results are joined in groups first
    (16, 1, "bf16", [16001]), (4, 1, "fp32", [40000]), (24, 2, "bf16", [9000, 1, 21000]), (8, 1, "bf16", [30000, 13, 9999]),
    (11, 1, "fp32", [700, 12000]),
]


@pytest.mark.parametrize("hq,hkv,dtype,lens", MANY_RUNS)
def test_attention_of_many_runs(hq, hkv, dtype, lens):
    B, scale = len(lens), 0.088
    p = _params(B, hq, hkv, dtype)
    blocks = -(-max(lens) // S)
    recs = _random_records(700, hkv, 141)
    bt = torch.randint(0, 700, (B, blocks), generator=_gen(142), device="cuda").int()
    Q = torch.randn((B, hq, D), generator=_gen(143), device="cuda").to(DT[dtype])
    O, lse, ws, err = _attn_buffers(B, hq, p)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = ice.Cache4(recs, bt)
    got = []
    for _ in range(4):  # the tickets of every call are those of the next one
        ice.ice_cache4_attn_decode(p, Q, cache, ln, scale, O, lse, ws, err)
        got.append((O.clone(), lse.clone()))
    assert ice.ice_check(err) == ice.ICE_OK
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])
    K, V = _rows_of(recs, bt, 0)
    _check_attn(O, lse, Q, lambda b, h: (K[b, h, :lens[b]], V[b, h, :lens[b]]), B, hkv, scale)
    # one after the other with a call of another shape in the same workspace
    p2, Q2 = _params(1, 32, 8, "bf16"), torch.randn((1, 32, D), generator=_gen(144), device="cuda").bfloat16()
    recs2, bt2 = _random_records(300, 8, 145), torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300)
    ln2 = torch.tensor([4700], dtype=torch.int32, device="cuda")
    ws = ice.workspace(max(ice.ice_attn4_workspace_bytes(x) for x in (p, p2)))
    O2, lse2, ws2, _ = _attn_buffers(1, 32, p2)
    ice.ice_cache4_attn_decode(p2, Q2, ice.Cache4(recs2, bt2), ln2, scale, O2, lse2, ws2, err)
    for _ in range(3):
        x, y = torch.empty_like(O), torch.empty_like(O2)
        ice.ice_cache4_attn_decode(p, Q, cache, ln, scale, x, None, ws, err)
        ice.ice_cache4_attn_decode(p2, Q2, ice.Cache4(recs2, bt2), ln2, scale, y, None, ws, err)
        assert torch.equal(x, got[0][0]) and torch.equal(y, O2)


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_attention_scales_and_values_that_are_not_numbers(scale):
    p = _params(1, 8, 1, "bf16")
    n = 100
    recs = _random_records(7, 1, 161)
    bt = torch.arange(7, dtype=torch.int32, device="cuda").view(1, 7)
    Q = torch.randn((1, 8, D), generator=_gen(162), device="cuda").bfloat16()
    O, lse, ws, err = _attn_buffers(1, 8, p)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, scale, O, lse, ws, err)
    K, V = _rows_of(recs, bt, 0)
    sign = -1 if scale < 0 else 1
    _check_attn(O, lse, sign * Q, lambda b, h: (K[b, h, :n], V[b, h, :n]), 1, 1, abs(scale))
    # one value group that is not a number: its half of O; one key: the whole row of every head
    recs[2, 0, 2176 + 8 * 5:2176 + 8 * 5 + 4] = 0xFF
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, scale, O, lse, ws, err)
    assert bool(O[..., :64].isnan().all()) and bool(O[..., 64:].isfinite().all())
    recs[2, 0, 1024:1028] = 0xFF
    ice.ice_cache4_attn_decode(p, Q, ice.Cache4(recs, bt), ln, scale, O, lse, ws, err)
    assert bool(O.isnan().all()) and bool(lse.isnan().all())
    assert ice.ice_check(err) == ice.ICE_OK
