"""Cases for the operators around the 4-bit paged cache.

rope    ice_qkv_rope             norms of q and k per head and the position rotation, from the projection's layout
append  ice_cache4_append        the same, with K and V into a token-ordered paged cache held in 4 bits
                                 (ice_cache4_read gives the values that the cache then holds)
attn    ice_cache4_attn_decode   attention of one query token a sequence over that cache
pack    ice_pool4_pack           a pool of semantic pages into 4-bit records (ice_pool4_unpack gives their values)
sparse  ice_sparse_attn_decode4  attention over selected pages of a 4-bit pool and a tail of new tokens

A 4-bit record holds 16 tokens of one KV head: K codes (1024 bytes), K (step, mid) pairs (128), V codes (1024),
V (step, mid) pairs (128).  A row of 128 is two groups of 64: step = bf16((max - min) / 15), mid = bf16((max + min) / 2),
code = clamp(rint((x - mid) / step + 7.5), 0, 15), value = mid + step * (code - 7.5).
"""
import math

import torch

own = False

D, S, G = 128, 16, 64  # head dimension, tokens a page, elements a group
KB, MB = S * D // 2, S * (D // G) * 4  # code bytes and (step, mid) bytes of K or V in a record
RECORD = 2 * (KB + MB)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of a Qwen3-32B-shaped batch: 16 single tokens, norms on q and k
        dict(name="rope_step_qwen3", op="rope", batch=16, tokens=1, hq=64, hkv=8, dtype="bf16", norm=True,
             interleaved=False, rotary=128, positions=131072),
        # a Mistral-7B-shaped prompt of 36k tokens
        dict(name="rope_prompt_mistral_36k", op="rope", batch=1, tokens=36864, hq=32, hkv=8, dtype="bf16", norm=False,
             interleaved=False, rotary=128, positions=40960),
        # one decode step of LongChat-7B-shaped sequences (as many KV heads as query heads) at about 100k tokens
        dict(name="append_step_longchat", op="append", batch=8, tokens=1, hq=32, hkv=32, dtype="bf16", norm=False,
             interleaved=False, rotary=128, positions=131072, start=99000),
        # four chunks of Llama-3.1-8B-shaped prompts, padded to the longest, starting inside a page
        dict(name="append_chunk_llama", op="append", batch=4, tokens=4099, hq=32, hkv=8, dtype="bf16", norm=False,
             interleaved=False, rotary=128, positions=16384, start=1237),
        # the tiny fp32 layout, adjacent pairs, half of the head rotated
        dict(name="append_tiny_fp32", op="append", batch=3, tokens=129, hq=4, hkv=1, dtype="fp32", norm=False,
             interleaved=True, rotary=64, positions=4096, start=5),
        # one Llama-3.1-8B-shaped sequence of 16k tokens: few units, split over the card
        dict(name="attn_llama_16k", op="attn", batch=1, hq=32, hkv=8, dtype="bf16", length=16384, ragged=False),
        # the Qwen3-32B-shaped batch at 100k tokens
        dict(name="attn_qwen3_100k", op="attn", batch=16, hq=64, hkv=8, dtype="bf16", length=100000, ragged=False),
        # many sequences of very different lengths, some empty
        dict(name="attn_ragged_b61", op="attn", batch=61, hq=32, hkv=8, dtype="bf16", length=4097, ragged=True),
        # a 16k Llama-3.1-8B-shaped layer's pool
        dict(name="pack_llama_16k", op="pack", units=8, pages=2017, dtype="bf16"),
        # a 100k LongChat-7B-shaped layer's pool
        dict(name="pack_longchat_100k", op="pack", units=32, pages=12487, dtype="bf16"),
        # the Qwen3-32B-shaped batch, budget 256: up to 128 pages a unit, and up to 300 new tokens a sequence
        dict(name="sparse_qwen3_100k", op="sparse", batch=16, hq=64, hkv=8, dtype="bf16", pages=11000, selected=128,
             tail=300),
        # one Mistral-7B-shaped sequence, budget 256, no tail
        dict(name="sparse_mistral_36k", op="sparse", batch=1, hq=32, hkv=8, dtype="bf16", pages=4300, selected=64,
             tail=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "pack", "sparse"])
    hq, hkv = rng.choice([(4, 1), (32, 8), (32, 32), (64, 8), (16, 1), (24, 2)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("rope", "append"):
        step = rng.random() < 0.4
        batch = _log(rng, 1, 64) if step else rng.randint(1, 4)
        tokens = rng.randint(1, 3) if step else _log(rng, 17, 6000)
        norm = rng.random() < 0.5 and (op == "rope" or dtype == "bf16")
        start = _log(rng, 1, 100000) - 1
        c = dict(op=op, batch=batch, tokens=tokens, hq=hq, hkv=hkv, dtype=dtype, norm=norm,
                 interleaved=rng.random() < 0.3, rotary=rng.choice([128, 128, 64, 96]), positions=start + tokens)
        return dict(c, start=start) if op == "append" else c
    if op == "attn":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype,
                    length=_log(rng, 1, max(2, min(100000, 6000000 // (batch * hkv)))), ragged=rng.random() < 0.6)
    if op == "pack":
        units = _log(rng, 1, 128)
        return dict(op=op, units=units, pages=_log(rng, 1, min(12000, 200000 // units)), dtype=dtype)
    return dict(op=op, batch=_log(rng, 1, 32), hq=hq, hkv=hkv, dtype=dtype, pages=_log(rng, 200, 4000),
                selected=_log(rng, 1, 200), tail=rng.choice([0, rng.randint(1, 700)]))


def _lengths(c, seed):
    """The tokens of each sequence (host): the same for prepare() and work()."""
    g = torch.Generator().manual_seed(seed)
    if c["op"] == "sparse":
        return torch.randint(0, c["tail"] + 1, (c["batch"],), generator=g) if c["tail"] else None
    n = torch.full((c["batch"],), c["length"])
    if c["ragged"]:
        n = torch.exp(torch.rand(c["batch"], generator=g) * math.log(c["length"] + 1)).long().clamp(max=c["length"])
        n[torch.rand(c["batch"], generator=g) < 0.05] = 0
    return n


def _selected(c, seed):
    """The selected pages of each unit (host)."""
    g = torch.Generator().manual_seed(seed + 1)
    most = min(c["selected"], c["pages"])
    return torch.randint((most + 1) // 2, most + 1, (c["batch"] * c["hkv"],), generator=g)


def _counts(c, seed):
    """The new tokens of each sequence (host): padded batches where a call appends more than one."""
    n = torch.full((c["batch"],), c["tokens"])
    if c["tokens"] > 1 and c["batch"] > 1:
        g = torch.Generator().manual_seed(seed + 2)
        n = torch.randint(c["tokens"] // 2, c["tokens"] + 1, (c["batch"],), generator=g)
        n[0] = c["tokens"]
    return n


def work(case):
    c = case
    if c["op"] == "pack":
        e = DTYPES[c["dtype"]].itemsize
        n = c["units"] * c["pages"]
        return {"bytes": n * (4 * S * D * e + 2 * RECORD), "flops": 16.0 * n * 2 * S * D}
    e = DTYPES[c["dtype"]].itemsize
    if c["op"] in ("rope", "append"):
        n = c["batch"] * c["tokens"]
        rows = c["hq"] + 2 * c["hkv"]
        b = n * (2 * rows * D * e + 4 * c["rotary"])
        if c["op"] == "append":
            n = int(_counts(c, 0).sum())
            b = n * (2 * rows * D * e + 4 * c["rotary"] + 2 * c["hkv"] * RECORD // S)
        return {"bytes": b, "flops": 8.0 * n * rows * D}
    tokens = int(_lengths(c, 0).sum()) * c["hkv"] if c["op"] == "attn" or c["tail"] else 0
    rows = tokens
    if c["op"] == "sparse":
        rows += int(_selected(c, 0).sum()) * 17 // 2  # pages hold 1 to 16 tokens
        tokens = rows
    io = c["batch"] * c["hq"] * D * (e + 4)
    return {"bytes": rows * RECORD // S + io, "flops": 4.0 * tokens * (c["hq"] // c["hkv"]) * D}


# ------------------------------------------------------------------ inputs --
def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda")


def _keys(lead, rows, gen, centres=64):
    """Keys of a Gaussian mixture: [lead, rows, D] in 32 bits."""
    mu = _rand((centres, D), gen)
    at = torch.randint(0, centres, (lead, rows), generator=gen, device="cuda")
    return mu[at] + 0.3 * _rand((lead, rows, D), gen)


def prepare(case, seed):
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": c, "plan": {}}
    if c["op"] in ("rope", "append"):
        B, T, hq, hkv, rd = c["batch"], c["tokens"], c["hq"], c["hkv"], c["rotary"]
        # the output of one projection: q, k and v of a token side by side
        qkv = _rand((B, T, hq + 2 * hkv, D), gen)
        if c["norm"]:
            qkv *= 3.0
            st["q_norm"] = (1 + 0.2 * _rand((D,), gen)).to(dt)
            st["k_norm"] = (1 + 0.2 * _rand((D,), gen)).to(dt)
        qkv = qkv.to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        inv = 1e6 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
        angle = torch.arange(c["positions"], dtype=torch.float64, device="cuda")[:, None] * inv
        st["table"] = torch.stack((angle.cos(), angle.sin()), -1).float()
        st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["q_out"] = torch.zeros((B, T, hq, D), dtype=dt, device="cuda")
        st["k_out"] = torch.zeros((B, hkv, T, D), dtype=dt, device="cuda")
        st["v_out"] = torch.zeros((B, hkv, T, D), dtype=dt, device="cuda")
        if c["op"] == "rope":
            first = torch.randint(0, c["positions"] - T + 1, (B, 1), generator=gen, device="cuda")
            st["positions"] = (first + torch.arange(T, device="cuda")).int()
            return st
        counts = _counts(c, seed).to("cuda")
        back = torch.randint(0, c["start"] + 1, (B,), generator=gen, device="cuda") // 64
        st["start"] = (c["start"] - back).int()
        st["counts"] = counts.int()
        blocks = -(-(c["start"] + T) // S)
        perm = torch.randperm(B * blocks, generator=gen, device="cuda")
        st["block_table"] = perm.view(B, blocks).int()
        st["records"] = torch.zeros((B * blocks, hkv, RECORD), dtype=torch.uint8, device="cuda")
        return st
    if c["op"] == "pack":
        U, P = c["units"], c["pages"]
        lens = torch.randint(1, S + 1, (U, P), generator=gen, device="cuda").int()
        used = (torch.arange(S, device="cuda") < lens[..., None])[..., None]
        st["pool_k"] = (_keys(U, P * S, gen).view(U, P, S, D) * used).to(dt)
        st["pool_v"] = (_rand((U, P, S, D), gen) * used).to(dt)
        st["page_len"] = lens
        st["n_pages"] = torch.full((U,), P, dtype=torch.int32, device="cuda")
        st["records"] = torch.zeros((U, P, RECORD), dtype=torch.uint8, device="cuda")
        st["k_out"], st["v_out"] = torch.zeros_like(st["pool_k"]), torch.zeros_like(st["pool_v"])
        st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return st
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    st["Q"] = _rand((B, hq, D), gen).to(dt)
    st["scale"] = 1.0 / math.sqrt(D)
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    st["O"] = torch.zeros((B, hq, D), dtype=torch.float32, device="cuda")
    st["lse"] = torch.zeros((B, hq), dtype=torch.float32, device="cuda")
    lens = _lengths(c, seed)
    st["lens"] = st["cache"] = st["block_table"] = None
    if lens is not None:
        blocks = max(1, -(-int(lens.max()) // S))
        st["lens"] = lens.to("cuda").int()
        st["block_table"] = torch.randperm(B * blocks, generator=gen, device="cuda").view(B, blocks).int()
        st["cache"] = _record_of(B * blocks * hkv, gen).view(B * blocks, hkv, RECORD)
    if c["op"] == "sparse":
        U, P = B * hkv, c["pages"]
        count = _selected(c, seed).to("cuda")
        most = min(c["selected"], P)
        pick = torch.rand((U, P), generator=gen, device="cuda").topk(most, dim=1).indices.sort(dim=1).values
        drop = torch.arange(most, device="cuda") >= count[:, None]
        st["sel_pages"] = pick.masked_fill(drop, -1).int()
        st["sel_count"] = count.int()
        st["page_len"] = torch.randint(1, S + 1, (U, P), generator=gen, device="cuda").int()
        st["records"] = _record_of(U * P, gen).view(U, P, RECORD)
    return st


def _record_of(n, gen):
    """n records of mixture keys and Gaussian values."""
    out = torch.empty((n, RECORD), dtype=torch.uint8, device="cuda")
    part = 1 << 17
    for i in range(0, n, part):
        m = min(part, n - i)
        k = _keys(1, m * S, gen).view(m, S, D).bfloat16()
        v = _rand((m, S, D), gen).bfloat16()
        out[i:i + m] = _write(k, v)
    return out


def _write(k, v):
    """Records [n, RECORD] of rows [n, S, D]."""
    n = k.shape[0]
    ck, mk = _codes(k)
    cv, mv = _codes(v)
    byte = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731  two codes a byte, the first in the low half
    # K: a row's sixteen 4-byte words (eight codes each), word 4 i + j at place 4 j + i
    kb = byte(ck).view(n, S, 4, 4, 4).transpose(2, 3).reshape(n, KB)
    # V: pieces of four codes (two bytes); piece 8 j + r of tokens 2 t, 2 t + 1 are the halves of word (t, r, j)
    vb = byte(cv).view(n, S // 2, 2, 4, 8, 2).permute(0, 1, 4, 3, 2, 5).reshape(n, KB)
    raw = lambda m: m.reshape(n, S * (D // G) * 2).bfloat16().view(torch.uint8)  # noqa: E731
    return torch.cat((kb, raw(mk), vb, raw(mv)), -1)


# ------------------------------------------------------------ plain forms --
def _codes(x):
    """Codes [..., D] (uint8) and (step, mid) [..., D / G, 2] of rows.  Differences and quotients of bf16 values are
    exact enough in 32 bits that no code changes; fp32 values next to a border between two codes take 64."""
    g = (x.double() if x.dtype == torch.float32 else x.float()).unflatten(-1, (D // G, G))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    step = ((hi - lo) / 15).float().bfloat16().float()
    mid = ((hi + lo) * 0.5).float().bfloat16().float()
    c = torch.round((g - mid) / step + 7.5).clamp(0, 15)
    c = torch.where(step == 0, torch.zeros_like(c), c)
    return c.flatten(-2).to(torch.uint8), torch.cat((step, mid), -1)


def _values(codes, meta):
    c = codes.float().unflatten(-1, (D // G, G))
    return (meta[..., 1:2] + meta[..., 0:1] * (c - 7.5)).flatten(-2)


def _read(rec):
    """K and V rows [..., S, D] in 32 bits of records [..., RECORD]."""
    lead = rec.shape[:-1]
    pair = lambda b: torch.stack((b & 15, b >> 4), -1).flatten(-2)  # noqa: E731
    meta = lambda b: b.contiguous().view(torch.bfloat16).float().view(*lead, S, D // G, 2)  # noqa: E731
    kb = rec[..., :KB].reshape(*lead, S, 4, 4, 4).transpose(-3, -2).reshape(*lead, S, D // 2)
    vb = rec[..., KB + MB:2 * KB + MB].reshape(*lead, S // 2, 8, 4, 2, 2)
    vb = vb.movedim(-2, -4).transpose(-3, -2).reshape(*lead, S, D // 2)
    k = _values(pair(kb), meta(rec[..., KB:KB + MB]))
    return k, _values(pair(vb), meta(rec[..., 2 * KB + MB:]))


def _norm(x, w, eps):
    ms = x.double().square().mean(-1, keepdim=True).float()
    r = (1 / (ms + eps).double().sqrt()).float()
    return (x * r) * w.float()


def _rotate(x, table, pos, c):
    """x [B, T, H, D] in 32 or 64 bits, positions [B, T]."""
    rd = c["rotary"]
    cs = table.to(x.dtype)[pos.clamp(0, table.shape[0] - 1).long()][:, :, None]
    cos, sin = cs[..., 0], cs[..., 1]
    if c["interleaved"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rd:]), -1)


def _plain_rows(st, pos):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    q, k = st["q"].float(), st["k"].float()
    if c["norm"]:
        q, k = _norm(q, st["q_norm"], 1e-6), _norm(k, st["k_norm"], 1e-6)
    if c["op"] == "append" and dt == torch.float32:
        k = k.double()  # a value next to a border between two codes
    return _rotate(q, st["table"], pos, c).to(dt), _rotate(k, st["table"], pos, c).to(dt)


def _plain_attention(Q, K, V, keep, scale):
    """Q [B, Hq, D], K and V [B, Hkv, L, D] in 32 bits, keep [B, Hkv, L]."""
    B, hq = Q.shape[:2]
    hkv = K.shape[1]
    q = Q.float().view(B, hkv, hq // hkv, D)
    s = (q @ K.transpose(-1, -2)) * scale
    s = s.masked_fill(~keep[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = (p @ torch.where(keep[..., None], V, torch.zeros_like(V))) / torch.where(l > 0, l, torch.ones_like(l))
    return o.reshape(B, hq, D), (m + torch.log(l)).reshape(B, hq)


def _cache_rows(st):
    c = st["case"]
    k, v = _read(st["cache"][st["block_table"].long()])  # [B, blocks, Hkv, S, D]
    B, blocks = st["block_table"].shape
    flat = lambda x: x.transpose(1, 2).reshape(B, c["hkv"], blocks * S, D)  # noqa: E731
    keep = torch.arange(blocks * S, device="cuda") < st["lens"][:, None]
    return flat(k), flat(v), keep[:, None].expand(B, c["hkv"], blocks * S)


def _plain(st):
    c = st["case"]
    if c["op"] == "rope":
        q, k = _plain_rows(st, st["positions"])
        return {"q": q, "k": k.transpose(1, 2).contiguous(), "v": st["v"].transpose(1, 2).contiguous()}
    if c["op"] == "append":
        t = torch.arange(c["tokens"], device="cuda")
        q, k = _plain_rows(st, st["start"][:, None] + t)
        new = (t < st["counts"][:, None])[..., None, None]
        held = lambda x: _values(*_codes(x)).to(x.dtype)  # noqa: E731
        clean = lambda x: torch.where(new, x, torch.zeros_like(x))  # noqa: E731
        return {"q": clean(q), "k": clean(held(k)).transpose(1, 2).contiguous(),
                "v": clean(held(st["v"])).transpose(1, 2).contiguous()}
    if c["op"] == "pack":
        used = (torch.arange(S, device="cuda") < st["page_len"][..., None])[..., None]
        held = lambda x: (_values(*_codes(x)) * used).to(x.dtype)  # noqa: E731
        return {"k": held(st["pool_k"]), "v": held(st["pool_v"])}
    if c["op"] == "attn":
        k, v, keep = _cache_rows(st)
        o, lse = _plain_attention(st["Q"], k, v, keep, st["scale"])
        return {"o": o, "lse": lse}
    B, hkv = c["batch"], c["hkv"]
    u = torch.arange(B * hkv, device="cuda")[:, None]
    at = st["sel_pages"].clamp(min=0).long()
    k, v = _read(st["records"][u, at])  # [U, max_sel, S, D]
    keep = torch.arange(S, device="cuda") < st["page_len"][u, at][..., None]
    keep &= (torch.arange(at.shape[1], device="cuda") < st["sel_count"][:, None])[..., None]
    k, v, keep = (x.reshape(B, hkv, -1, *x.shape[3:]) for x in (k, v, keep))
    if st["lens"] is not None:
        tk, tv, tkeep = _cache_rows(st)
        k, v, keep = torch.cat((k, tk), 2), torch.cat((v, tv), 2), torch.cat((keep, tkeep), 2)
    o, lse = _plain_attention(st["Q"], k, v, keep, st["scale"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------- the framework's --
def _plan(st):
    """What a program keeps beside its buffers: the parameters, the views and the workspace."""
    import semantic_paged_kv_gb300 as ice

    c, pl = st["case"], {}
    dtype = ice.ICE_BF16 if c["dtype"] == "bf16" else ice.ICE_FP32
    if c["op"] == "pack":
        cfg = ice.Config(batch=1, n_q_heads=c["units"], n_kv_heads=c["units"], n_tokens=0, dtype=dtype,
                         np_cap=1, page_cap=c["pages"])
        pl["index"] = ice.IceIndex(n_pages=st["n_pages"].data_ptr(), page_len=st["page_len"].data_ptr(),
                                   pool_k=st["pool_k"].data_ptr(), pool_v=st["pool_v"].data_ptr())
        pl["out"] = ice.IceIndex(n_pages=st["n_pages"].data_ptr(), page_len=st["page_len"].data_ptr(),
                                 pool_k=st["k_out"].data_ptr(), pool_v=st["v_out"].data_ptr())
    else:
        cfg = ice.Config(batch=c["batch"], n_q_heads=c["hq"], n_kv_heads=c["hkv"], n_tokens=0, dtype=dtype, np_cap=1,
                         page_cap=c.get("pages", 1))
    pl["params"] = cfg.params()
    if c["op"] in ("rope", "append"):
        for f in ("q", "k", "v", "q_out"):
            pl[f] = ice.rows(st[f])
        for f in ("k_out", "v_out"):
            pl[f] = ice.rows(st[f].transpose(1, 2))
        pl["rope"] = ice.Rope(st["table"], interleaved=c["interleaved"], q_norm=st.get("q_norm"),
                              k_norm=st.get("k_norm"), eps=1e-6)
    if c["op"] == "append":
        pl["cache"] = ice.Cache4(st["records"], st["block_table"])
    if c["op"] in ("attn", "sparse"):
        pl["cache"] = None if st["cache"] is None else ice.Cache4(st["cache"], st["block_table"])
        pl["ws"] = ice.workspace(ice.ice_attn4_workspace_bytes(pl["params"]))
    return pl


def _framework(st):
    import semantic_paged_kv_gb300 as ice

    c = st["case"]
    pl = st["plan"]
    if not pl:
        pl.update(_plan(st))
    if c["op"] == "rope":
        ice.ice_qkv_rope(pl["params"], c["tokens"], pl["q"], pl["k"], pl["v"], st["positions"], None, None, pl["rope"],
                         pl["q_out"], pl["k_out"], pl["v_out"], st["err"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    if c["op"] == "append":
        ice.ice_cache4_append(pl["params"], c["tokens"], pl["q"], pl["k"], pl["v"], None, st["start"], st["counts"],
                              pl["rope"], pl["q_out"], pl["cache"], st["err"])
        ice.ice_cache4_read(pl["params"], c["tokens"], pl["cache"], st["start"], st["counts"], pl["k_out"],
                            pl["v_out"], st["err"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    if c["op"] == "pack":
        ice.ice_pool4_pack(pl["params"], pl["index"], 0, st["records"], st["err"])
        ice.ice_pool4_unpack(pl["params"], pl["out"], st["records"], st["err"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if c["op"] == "attn":
        ice.ice_cache4_attn_decode(pl["params"], st["Q"], pl["cache"], st["lens"], st["scale"], st["O"], st["lse"],
                                   pl["ws"], st["err"])
    else:
        ice.ice_sparse_attn_decode4(pl["params"], st["Q"], st["records"], st["page_len"], st["sel_pages"],
                                    st["sel_count"], pl["cache"], st["lens"], st["scale"], st["O"], st["lse"],
                                    pl["ws"], st["err"])
    return {"o": st["O"], "lse": st["lse"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ exact --
def _exact_held(x, lens_ok):
    """What 4 bits hold of rows in 64 bits; zero where lens_ok is false."""
    a, b = x[..., :G], x[..., G:]
    parts = []
    for h in (a, b):
        lo, hi = h.min(-1, keepdim=True).values, h.max(-1, keepdim=True).values
        step = ((hi - lo) / 15).float().bfloat16().double()
        mid = ((hi + lo) / 2).float().bfloat16().double()
        n = torch.clamp(torch.round((h - mid) / torch.where(step > 0, step, torch.ones_like(step)) + 7.5), 0, 15)
        parts.append(torch.where(step > 0, mid + step * (n - 7.5), mid))
    return torch.where(lens_ok, torch.cat(parts, -1), torch.zeros_like(x))


def _exact_record(rec):
    """K and V [n, S, D] in 64 bits of records [n, RECORD], each element looked up at its own place."""
    d = torch.arange(D, device=rec.device)
    t = torch.arange(S, device=rec.device)[:, None]
    w = d // 8
    kat = t * 64 + ((w % 4) * 4 + w // 4) * 4 + (d % 8) // 2
    piece = d // 4
    vat = KB + MB + (((t // 2) * 8 + piece % 8) * 4 + piece // 8) * 4 + (t % 2) * 2 + (d % 4) // 2
    got = []
    for at, meta in ((kat, KB), (vat, 2 * KB + MB)):
        code = (rec[:, at].int() >> (4 * (d % 2))) & 15
        pair = rec[:, meta:meta + MB].contiguous().view(torch.bfloat16).double().view(-1, S, D // G, 2)
        pair = pair.repeat_interleave(G, dim=2)
        got.append(pair[..., 1] + pair[..., 0] * (code.double() - 7.5))
    return got


def _exact_attention(q, k, v, scale):
    """One sequence's KV head: q [g, D], k and v [L, D] in 64 bits."""
    if not k.shape[0]:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    s = (q @ k.T) * scale
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]) @ v, lse


def _exact_rows(st, pos):
    c = st["case"]
    rd = c["rotary"]
    z = torch.view_as_complex(st["table"].double())[pos.long()][:, :, None]
    out = []
    for x, w in ((st["q"], st.get("q_norm")), (st["k"], st.get("k_norm"))):
        x = x.double()
        if c["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        if c["interleaved"]:
            y = torch.view_as_real(torch.view_as_complex(x[..., :rd].unflatten(-1, (rd // 2, 2)).contiguous()) * z)
            y = y.flatten(-2)
        else:
            y = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * z
            y = torch.cat((y.real, y.imag), -1)
        out.append(torch.cat((y, x[..., rd:]), -1))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] in ("rope", "append"):
        t = torch.arange(c["tokens"], device="cuda")
        pos = st["positions"] if c["op"] == "rope" else st["start"][:, None] + t
        q, k = _exact_rows(st, pos)
        if c["op"] == "rope":
            return {"q": q, "k": k.transpose(1, 2).contiguous(), "v": st["v"].double().transpose(1, 2).contiguous()}
        new = (t < st["counts"][:, None])[..., None, None]
        dt = DTYPES[c["dtype"]]
        hold = lambda x: _exact_held(x, new).transpose(1, 2).contiguous()  # noqa: E731
        # the cache holds what the storage type would hold, in 4 bits
        return {"q": torch.where(new, q, torch.zeros_like(q)), "k": hold(k.to(dt).double()), "v": hold(st["v"].double())}
    if c["op"] == "pack":
        used = (torch.arange(S, device="cuda") < st["page_len"][..., None])[..., None]
        return {"k": _exact_held(st["pool_k"].double(), used), "v": _exact_held(st["pool_v"].double(), used)}
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    g = hq // hkv
    o = torch.zeros((B, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(hkv):
            k, v = [], []
            if c["op"] == "sparse":
                u = b * hkv + h
                at = st["sel_pages"][u, :int(st["sel_count"][u])].long()
                ok = torch.arange(S, device="cuda") < st["page_len"][u, at][:, None]
                for x, y in zip((k, v), _exact_record(st["records"][u, at])):
                    x.append(y[ok])
            if st["lens"] is not None:
                n = int(st["lens"][b])
                at = st["block_table"][b, :-(-n // S)].long()
                for x, y in zip((k, v), _exact_record(st["cache"][at, h])):
                    x.append(y.reshape(-1, D)[:n])
            hs = slice(h * g, (h + 1) * g)
            o[b, hs], lse[b, hs] = _exact_attention(st["Q"][b, hs].double(), torch.cat(k), torch.cat(v), st["scale"])
    return {"o": o, "lse": lse}
