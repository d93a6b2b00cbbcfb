"""Cases for the operators that verify trees of drafted tokens over the 4-bit pages.

tree    ice_cache4_attn_tree    attention of a sequence's drafted tokens over its 4-bit cache and over one another: a
                                node sees the cache, its ancestors and itself; without parents a chain of new tokens
sparse  ice_sparse_attn_tree4   the same over selected pages of a 4-bit pool, a cache of new tokens and the tree
verify  ice_tree_verify         which drafted tokens the target model accepts, from given random numbers
commit  ice_cache4_commit       the accepted nodes' keys and values into the 4-bit caches of all layers
                                (ice_cache4_read gives the values that the caches then hold)

A 4-bit record holds 16 tokens of one KV head: K codes (1024 bytes), K (step, mid) pairs (128), V codes (1024),
V (step, mid) pairs (128).  A row of 128 is two groups of 64: step = bf16((max - min) / 15), mid = bf16((max + min) / 2),
code = clamp(rint((x - mid) / step + 7.5), 0, 15), value = mid + step * (code - 7.5).

Verification starts at node 0, the last token that the target model has accepted.  At node i with the target's
probabilities p = target[i] and the draft's q = draft[i], the children c of i (parents[c] = i) are tried in order, with
rest = max(p - beta q, 0) and mass the sum of rest, at first beta = 0 and mass = 1: child c with token x is accepted if
uniform[c] q(x) mass < p(x) - beta q(x), and its own children are tried next; otherwise beta grows by mass.  Where no
child is left, the next token is the first x with sum_{y <= x} rest(y) > uniform[0] sum rest.  Without draft
probabilities (each drafted token is certain) c is accepted if uniform[c] mass < p(x); otherwise p(x) is left out from
then on and mass falls by it.  Without random numbers a child is accepted if it is the target's likeliest token.
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
        # one speculative step of a Llama-3.1-8B-shaped sequence at 16k tokens, a tree of 26 nodes
        dict(name="tree_llama_16k", op="tree", batch=1, hq=32, hkv=8, dtype="bf16", nodes=26, tree=True, length=16384,
             ragged=False),
        # the Qwen3-32B-shaped batch at 100k tokens, 16 nodes a sequence
        dict(name="tree_qwen3_100k", op="tree", batch=16, hq=64, hkv=8, dtype="bf16", nodes=16, tree=True,
             length=100000, ragged=False),
        # LongChat-7B-shaped heads (one query head a KV head), large trees, very different lengths, some empty
        dict(name="tree_longchat_ragged", op="tree", batch=9, hq=32, hkv=32, dtype="bf16", nodes=61, tree=True,
             length=20001, ragged=True),
        # a chunk of 1000 new tokens of a Mistral-7B-shaped prompt behind 36k tokens
        dict(name="chunk_mistral_36k", op="tree", batch=1, hq=32, hkv=8, dtype="bf16", nodes=1000, tree=False,
             length=36864, ragged=False),
        # the tiny fp32 layout
        dict(name="tree_tiny_fp32", op="tree", batch=3, hq=4, hkv=1, dtype="fp32", nodes=7, tree=True, length=2048,
             ragged=True),
        # the Qwen3-32B-shaped batch, up to 128 selected pages a unit, up to 300 new tokens and a tree a sequence
        dict(name="sparse_tree_qwen3", op="sparse", batch=16, hq=64, hkv=8, dtype="bf16", nodes=16, tree=True,
             pages=11000, selected=128, tail=300),
        # one Mistral-7B-shaped sequence, selected pages and a chain of five drafted tokens
        dict(name="sparse_chain_mistral", op="sparse", batch=1, hq=32, hkv=8, dtype="bf16", nodes=5, tree=False,
             pages=4300, selected=64, tail=0),
        # one sequence, a tree of 26 nodes
        dict(name="verify_step", op="verify", batch=1, nodes=26, vocab=128000, dtype="fp32", mode="sample"),
        # a batch of 64 sequences with trees of up to 61 nodes, probabilities in bf16
        dict(name="verify_batch", op="verify", batch=64, nodes=61, vocab=128000, dtype="bf16", mode="sample"),
        # drafted tokens without probabilities (the draft's likeliest ones), a small odd vocabulary
        dict(name="verify_certain", op="verify", batch=16, nodes=26, vocab=32003, dtype="fp32", mode="certain"),
        # one speculative step's accepted tokens into the caches of 32 Llama-3.1-8B-shaped layers
        dict(name="commit_llama", op="commit", layers=32, batch=1, hkv=8, dtype="bf16", nodes=26, start=16384),
        # the same for the Qwen3-32B-shaped batch, 64 layers
        dict(name="commit_qwen3", op="commit", layers=64, batch=16, hkv=8, dtype="bf16", nodes=16, start=4099),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "sparse", "verify", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "verify":
        mode = rng.choice(["sample", "sample", "certain", "greedy"])
        return dict(op=op, batch=_log(rng, 1, 64), nodes=_log(rng, 1, 61), vocab=_log(rng, 1000, 128000), dtype=dtype,
                    mode=mode)
    hq, hkv = rng.choice([(4, 1), (32, 8), (32, 32), (64, 8), (16, 1), (24, 2)])
    if op == "commit":
        batch = _log(rng, 1, 16)
        return dict(op=op, layers=_log(rng, 1, 64), batch=batch, hkv=min(hkv, 8), dtype=dtype, nodes=_log(rng, 1, 64),
                    start=_log(rng, 1, 4100) - 1)
    tree = rng.random() < 0.7
    nodes = _log(rng, 1, 128) if tree else _log(rng, 1, 1000)
    if dtype == "fp32":
        nodes = min(nodes, 61)
    if op == "sparse":
        batch = _log(rng, 1, 16)
        nodes = min(nodes, 4000 // batch)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, nodes=nodes, tree=tree,
                    pages=_log(rng, 200, 4000), selected=_log(rng, 1, 200), tail=rng.choice([0, rng.randint(1, 700)]))
    batch = _log(rng, 1, 32)
    nodes = min(nodes, 4000 // batch)
    most = 6000000 // (batch * hkv) if dtype == "bf16" else 200000 // (batch * hkv)
    most = min(100000, most, 1000000000 // (batch * hq * nodes))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, nodes=nodes, tree=tree,
                length=_log(rng, 1, max(2, most)), ragged=rng.random() < 0.6)


def _lengths(c, seed):
    """The cached tokens of each sequence (host): the same for prepare() and work()."""
    g = torch.Generator().manual_seed(seed)
    if c["op"] == "sparse":
        return torch.randint(0, c["tail"] + 1, (c["batch"],), generator=g) if c["tail"] else None
    n = torch.full((c["batch"],), c["length"])
    if c["ragged"]:
        n = torch.exp(torch.rand(c["batch"], generator=g) * math.log(c["length"] + 1)).long().clamp(max=c["length"])
        n[torch.rand(c["batch"], generator=g) < 0.1] = 0
    return n


def _selected(c, seed):
    """The selected pages of each unit (host)."""
    g = torch.Generator().manual_seed(seed + 1)
    most = min(c["selected"], c["pages"])
    return torch.randint((most + 1) // 2, most + 1, (c["batch"] * c["hkv"],), generator=g)


def _counts(c, seed):
    """The nodes of each sequence (host): padded batches."""
    n = torch.full((c["batch"],), c["nodes"])
    if c["nodes"] > 1 and c["batch"] > 1:
        g = torch.Generator().manual_seed(seed + 2)
        n = torch.randint(c["nodes"] // 2, c["nodes"] + 1, (c["batch"],), generator=g)
        n[0] = c["nodes"]
    return n


def _parents(c, seed):
    """Parents [batch, nodes] (host): node 0 is the root; a later node hangs on one of the half before it."""
    g = torch.Generator().manual_seed(seed + 3)
    t = torch.arange(c["nodes"])
    low = (t - 1) // 3
    u = torch.rand((c["batch"], c["nodes"]), generator=g)
    return (low + (u * (t - low)).long()).clamp(max=t - 1).int()


def _paths(c, seed):
    """Accepted paths [batch, nodes] (-1 behind) and their lengths (host): a walk from the root to a node at random."""
    g = torch.Generator().manual_seed(seed + 4)
    parents = _parents(c, seed).tolist()
    path, n = torch.full((c["batch"], c["nodes"]), -1, dtype=torch.int32), []
    for b in range(c["batch"]):
        at, walk = int(torch.randint(0, c["nodes"], (1,), generator=g)), []
        while at >= 0:
            walk.append(at)
            at = parents[b][at]
        path[b, :len(walk)] = torch.tensor(walk[::-1], dtype=torch.int32)
        n.append(len(walk))
    return path, torch.tensor(n, dtype=torch.int32)


def work(case):
    c = case
    e = DTYPES[c["dtype"]].itemsize
    if c["op"] == "verify":
        # the rows of the last node at least
        rows = 2 if c["mode"] == "sample" else 1
        return {"bytes": c["batch"] * (rows * c["vocab"] * e + 12 * c["nodes"]),
                "flops": float(c["batch"] * rows * c["vocab"])}
    if c["op"] == "commit":
        n = int(_paths(c, 0)[1].sum()) * c["layers"] * c["hkv"]
        return {"bytes": n * (2 * D * e + RECORD // S + 2 * D * e + RECORD // S), "flops": 16.0 * n * 2 * D}
    counts = _counts(c, 0)
    lens = _lengths(c, 0)
    held = lens * c["hkv"] if lens is not None else torch.zeros(c["batch"], dtype=torch.long)  # over a sequence's heads
    if c["op"] == "sparse":
        held = held + _selected(c, 0).view(c["batch"], c["hkv"]).sum(1) * 17 // 2  # pages hold 1 to 16 tokens
    new = int(counts.sum())
    own_pairs = float((counts * (counts + 1) // 2).sum()) if not c["tree"] else float(counts.sum()) * 8
    pairs = float((held * counts).sum()) + own_pairs * c["hkv"]
    return {"bytes": int(held.sum()) * RECORD // S + new * (2 * c["hq"] + 2 * c["hkv"]) * D * e,
            "flops": 4.0 * pairs * (c["hq"] // c["hkv"]) * D}


# ------------------------------------------------------------------ inputs --
def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda")


def _keys(lead, rows, gen, centres=64):
    """Keys of a Gaussian mixture: [lead, rows, D] in 32 bits."""
    mu = _rand((centres, D), gen)
    at = torch.randint(0, centres, (lead, rows), generator=gen, device="cuda")
    return mu[at] + 0.3 * _rand((lead, rows, D), gen)


def _prepare_verify(c, st, gen, seed):
    dt = DTYPES[c["dtype"]]
    B, T, V = c["batch"], c["nodes"], c["vocab"]
    logits = 2.5 * _rand((B, T, V), gen)
    st["target"] = torch.softmax(logits, -1).to(dt)
    logits += 0.7 * _rand((B, T, V), gen)
    st["draft"] = torch.softmax(logits, -1).to(dt)
    parents = st["parents"].long().clamp(min=0)
    q = st["draft"].gather(1, parents[..., None].expand(B, T, V)).float() if B * T * V < 1 << 28 else None
    if q is None:  # a sequence at a time: the rows of all nodes' parents
        q = st["draft"]
        tokens = torch.stack([(q[b][parents[b]].float() / torch.empty((T, V), device="cuda").exponential_(
            generator=gen)).argmax(-1) for b in range(B)])
    elif c["mode"] == "sample":
        tokens = (q / torch.empty_like(q).exponential_(generator=gen)).argmax(-1)
    else:  # the draft's likeliest tokens, one for each of a node's children
        rank = (st["parents"][:, :, None] == st["parents"][:, None, :]).tril(-1).sum(-1)
        tokens = q.topk(min(T, V), -1).indices.gather(-1, rank[..., None].clamp(max=V - 1))[..., 0]
    st["tokens"] = tokens.int()
    st["uniform"] = torch.rand((B, T), generator=gen, device="cuda")
    if c["mode"] != "sample":
        st["draft"] = None
    if c["mode"] == "greedy":
        st["uniform"] = None
    st["path"] = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    st["n_path"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    st["next"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": c, "plan": {}, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    B, T = c["batch"], c["nodes"]
    st["counts"] = _counts(c, seed).int().to("cuda")
    st["parents"] = _parents(c, seed).to("cuda") if c.get("tree", True) else None
    if c["op"] == "verify":
        return _prepare_verify(c, st, gen, seed)
    hkv = c["hkv"]
    if c["op"] == "commit":
        L = c["layers"]
        st["k"], st["v"] = (_keys(L * B, T * hkv, gen).view(L, B, T, hkv, D).to(dt) for _ in range(2))
        path, n = _paths(c, seed)
        st["path"], st["n_path"] = path.to("cuda"), n.to("cuda")
        back = torch.randint(0, c["start"] + 1, (B,), generator=gen, device="cuda") // 64
        st["start"] = (c["start"] - back).int()
        blocks = -(-(c["start"] + T) // S)
        # every layer has pages of its own, in one array, under the same table
        st["block_table"] = torch.randperm(B * blocks, generator=gen, device="cuda").view(B, blocks).int()
        st["records"] = torch.zeros((L, B * blocks, hkv, RECORD), dtype=torch.uint8, device="cuda")
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
        return st
    hq = c["hq"]
    # the output of one projection: q, k and v of a token side by side
    qkv = _rand((B, T, hq + 2 * hkv, D), gen)
    qkv[:, :, hq:hq + hkv] = _keys(B, T * hkv, gen).view(B, T, hkv, D)
    qkv = qkv.to(dt)
    st["q"], st["k"], st["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    st["scale"] = 1.0 / math.sqrt(D)
    st["O"] = torch.zeros((B, T, hq, D), dtype=dt, device="cuda")
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


def _ancestors(st):
    """[B, T, T]: whether a node sees another one, itself among them."""
    T = st["case"]["nodes"]
    if st["parents"] is None:
        return torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(st["case"]["batch"], T, T)
    t = torch.arange(T, device="cuda")
    # every node's parent, and its parent's parent, ...: powers of the parents' matrix by squaring
    up = (st["parents"][:, :, None] == t).float() + torch.eye(T, device="cuda")
    for _ in range(max(1, T.bit_length())):
        up = ((up @ up) > 0).float()
    return up > 0


def _cache_rows(st):
    c = st["case"]
    k, v = _read(st["cache"][st["block_table"].long()])  # [B, blocks, Hkv, S, D]
    B, blocks = st["block_table"].shape
    flat = lambda x: x.transpose(1, 2).reshape(B, c["hkv"], blocks * S, D)  # noqa: E731
    keep = torch.arange(blocks * S, device="cuda") < st["lens"][:, None]
    return flat(k), flat(v), keep[:, None].expand(B, c["hkv"], blocks * S)


def _plain_tree(st):
    c = st["case"]
    B, T, hq, hkv = c["batch"], c["nodes"], c["hq"], c["hkv"]
    g = hq // hkv
    parts = []
    if c["op"] == "sparse":
        u = torch.arange(B * hkv, device="cuda")[:, None]
        at = st["sel_pages"].clamp(min=0).long()
        k, v = _read(st["records"][u, at])  # [U, max_sel, S, D]
        keep = torch.arange(S, device="cuda") < st["page_len"][u, at][..., None]
        keep &= (torch.arange(at.shape[1], device="cuda") < st["sel_count"][:, None])[..., None]
        parts.append([x.reshape(B, hkv, -1, *x.shape[3:]) for x in (k, v, keep)])
    if st["lens"] is not None:
        parts.append(_cache_rows(st))
    live = torch.arange(T, device="cuda") < st["counts"][:, None]
    q = st["q"].float().view(B, T, hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * T, D)
    tk, tv = (x.float().transpose(1, 2) for x in (st["k"], st["v"]))
    sees = _ancestors(st)[:, None, None].expand(B, hkv, g, T, T).reshape(B, hkv, g * T, T)
    s = [((q @ k.transpose(-1, -2)) * st["scale"]).masked_fill(~keep[:, :, None], -math.inf) for k, _, keep in parts]
    s.append(((q @ tk.transpose(-1, -2)) * st["scale"]).masked_fill(~sees, -math.inf))
    m = torch.stack([x.amax(-1, keepdim=True) for x in s if x.shape[-1]]).amax(0)
    o = torch.zeros((B, hkv, g * T, D), device="cuda")
    l = torch.zeros((B, hkv, g * T, 1), device="cuda")
    for x, v in zip(s, [v for _, v, _ in parts] + [tv]):
        p = torch.exp(x.sub_(m))
        l += p.sum(-1, keepdim=True)
        o += p @ v
    o = (o / l).view(B, hkv, g, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, hq, D)
    return {"o": (o * live[..., None, None]).to(DTYPES[c["dtype"]])}


def _plain_verify(st):
    c = st["case"]
    B, T, V = c["batch"], c["nodes"], c["vocab"]
    rows = torch.arange(B, device="cuda")
    node = torch.zeros(B, dtype=torch.long, device="cuda")
    n = torch.ones(B, dtype=torch.long, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    beta = torch.zeros((B, 1), dtype=torch.float64, device="cuda")
    mass = torch.ones((B, 1), dtype=torch.float64, device="cuda")
    p = st["target"][:, 0].double()
    q = st["draft"][:, 0].double() if st["draft"] is not None else None
    # nodes in order: a node's children come behind it, so one pass meets all that is tried
    for t in range(1, T):
        child = ((st["parents"][:, t] == node) & (t < st["counts"]))[:, None]
        x = st["tokens"][:, t].long()[:, None]
        px = p.gather(1, x)
        if c["mode"] == "greedy":
            take = child & (p.argmax(-1, keepdim=True) == x)
        elif q is None:
            take = child & (st["uniform"][:, t:t + 1].double() * mass < px)
            no = child & ~take
            mass = torch.where(no, (mass - px).clamp(min=0), mass)
            p = p.scatter(1, x, torch.where(no, torch.zeros_like(px), px))
        else:
            qx = q.gather(1, x)
            take = child & (st["uniform"][:, t:t + 1].double() * qx * mass < px - beta * qx)
            no = child & ~take
            beta = torch.where(no, beta + mass, beta)
            mass = torch.where(no, (p - beta * q).clamp(min=0).sum(-1, keepdim=True), mass)
        path.scatter_(1, n[:, None].clamp(max=T - 1),
                      torch.where(take, t, path.gather(1, n[:, None].clamp(max=T - 1))).int())
        node = torch.where(take[:, 0], t, node)
        n += take[:, 0]
        p = torch.where(take, st["target"][rows, t].double(), p)
        if q is not None:
            q = torch.where(take, st["draft"][rows, t].double(), q)
        beta, mass = torch.where(take, torch.zeros_like(beta), beta), torch.where(take, torch.ones_like(mass), mass)
    if c["mode"] == "greedy":
        nxt = p.argmax(-1)
    else:
        rest = p if q is None else (p - beta * q).clamp(min=0)
        rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, st["target"][rows, node].double())
        run = rest.cumsum(-1)
        nxt = (run > st["uniform"][:, :1].double() * run[:, -1:]).int().argmax(-1)
    return {"path": path, "n": n.int(), "next": nxt.int()}


def _plain_commit(st):
    c = st["case"]
    L, B, T = c["layers"], c["batch"], c["nodes"]
    at = st["path"].clamp(min=0).long()[None, :, :, None, None]
    new = (torch.arange(T, device="cuda") < st["n_path"][:, None])[None, :, :, None, None]
    out = {}
    for f in ("k", "v"):
        x = st[f].gather(2, at.expand(L, B, T, c["hkv"], D))
        out[f] = torch.where(new, _values(*_codes(x)).to(x.dtype), torch.zeros_like(x))
    return out


def _plain(st):
    op = st["case"]["op"]
    return _plain_verify(st) if op == "verify" else _plain_commit(st) if op == "commit" else _plain_tree(st)


# ------------------------------------------------------- the framework's --
def _plan(st):
    """What a program keeps beside its buffers: the parameters, the views, the workspace and buffers that a call fills."""
    import semantic_paged_kv_gb300 as ice

    c, pl = st["case"], {}
    pl["dtype"] = dtype = ice.ICE_BF16 if c["dtype"] == "bf16" else ice.ICE_FP32
    pl["tree"] = ice.Tree(st["parents"], st["counts"], c["nodes"])
    if c["op"] == "verify":
        pl["target"] = ice.probs(st["target"])
        pl["draft"] = None if st["draft"] is None else ice.probs(st["draft"])
        return pl
    L = c.get("layers", 1)
    config = lambda batch: ice.Config(batch=batch, n_q_heads=c.get("hq", c["hkv"]), n_kv_heads=c["hkv"],  # noqa: E731
                                      n_tokens=0, dtype=dtype, np_cap=1, page_cap=c.get("pages", 1)).params()
    pl["params"] = config(c["batch"])
    if c["op"] == "commit":
        pl["k"], pl["v"] = ice.rows(st["k"][0]), ice.rows(st["v"][0])
        pl["cache"] = ice.Cache4(st["records"][0], st["block_table"])
        # all layers as one cache, to read them back in one call: buffers that every call fills
        pages = st["records"].shape[1]
        pl["first"] = torch.arange(L, dtype=torch.int32, device="cuda")[:, None, None] * pages
        pl["all_table"] = torch.empty((L, *st["block_table"].shape), dtype=torch.int32, device="cuda")
        pl["all"] = ice.Cache4(st["records"].view(L * pages, c["hkv"], RECORD), pl["all_table"].flatten(0, 1))
        pl["all_params"] = config(L * c["batch"])
        pl["all_start"], pl["all_n"] = (torch.empty((L, c["batch"]), dtype=torch.int32, device="cuda") for _ in range(2))
        pl["out"] = torch.empty((2, *st["k"].shape), dtype=st["k"].dtype, device="cuda")
        st["k_out"], st["v_out"] = pl["out"]
        for f in ("k_out", "v_out"):
            pl[f] = ice.rows(st[f].view(L * c["batch"], c["nodes"], c["hkv"], D))
        return pl
    for f in ("q", "k", "v", "O"):
        pl[f] = ice.rows(st[f])
    pl["cache"] = None if st["cache"] is None else ice.Cache4(st["cache"], st["block_table"])
    pl["ws"] = ice.workspace(ice.ice_tree_workspace_bytes(pl["params"]))
    return pl


def _framework(st):
    import semantic_paged_kv_gb300 as ice

    c, pl = st["case"], st["plan"]
    if not pl:
        pl.update(_plan(st))
    if c["op"] == "tree":
        ice.ice_cache4_attn_tree(pl["params"], pl["tree"], pl["q"], pl["cache"], st["lens"], pl["k"], pl["v"],
                                 st["scale"], pl["O"], pl["ws"], st["err"])
        return {"o": st["O"]}
    if c["op"] == "sparse":
        ice.ice_sparse_attn_tree4(pl["params"], pl["tree"], pl["q"], st["records"], st["page_len"], st["sel_pages"],
                                  st["sel_count"], pl["cache"], st["lens"], pl["k"], pl["v"], st["scale"], pl["O"],
                                  pl["ws"], st["err"])
        return {"o": st["O"]}
    if c["op"] == "verify":
        ice.ice_tree_verify(pl["tree"], pl["target"], pl["draft"], st["tokens"], st["uniform"], st["path"],
                            st["n_path"], st["next"], st["err"])
        return {"path": st["path"], "n": st["n_path"], "next": st["next"]}
    ice.ice_cache4_commit(pl["params"], c["layers"], c["nodes"], pl["k"], pl["v"], st["path"], st["n_path"],
                          st["start"], pl["cache"], st["err"], k_layer=st["k"].stride(0), v_layer=st["v"].stride(0),
                          records_layer=st["records"].stride(0))
    torch.add(st["block_table"], pl["first"], out=pl["all_table"])
    pl["all_start"].copy_(st["start"])
    pl["all_n"].copy_(st["n_path"])
    pl["out"].zero_()  # (rows behind the path are not written)
    ice.ice_cache4_read(pl["all_params"], c["nodes"], pl["all"], pl["all_start"], pl["all_n"], pl["k_out"],
                        pl["v_out"], st["err"])
    return {"k": st["k_out"], "v": st["v_out"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ exact --
def _exact_held(x):
    """What 4 bits hold of rows in 64 bits."""
    parts = []
    for h in (x[..., :G], x[..., G:]):
        lo, hi = h.min(-1, keepdim=True).values, h.max(-1, keepdim=True).values
        step = ((hi - lo) / 15).float().bfloat16().double()
        mid = ((hi + lo) / 2).float().bfloat16().double()
        n = torch.clamp(torch.round((h - mid) / torch.where(step > 0, step, torch.ones_like(step)) + 7.5), 0, 15)
        parts.append(torch.where(step > 0, mid + step * (n - 7.5), mid))
    return torch.cat(parts, -1)


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


def _exact_tree(st):
    c = st["case"]
    B, T, hq, hkv = c["batch"], c["nodes"], c["hq"], c["hkv"]
    g = hq // hkv
    out = torch.zeros((B, T, hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["counts"][b])
        if not n:
            continue
        sees = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):  # a node sees what its parent sees, and itself
            up = i - 1 if st["parents"] is None else int(st["parents"][b, i])
            if up >= 0:
                sees[i] = sees[up]
            sees[i, i] = True
        sees = sees.to("cuda")
        for h in range(hkv):
            k, v = [], []
            if c["op"] == "sparse":
                u = b * hkv + h
                at = st["sel_pages"][u, :int(st["sel_count"][u])].long()
                ok = torch.arange(S, device="cuda") < st["page_len"][u, at][:, None]
                for x, y in zip((k, v), _exact_record(st["records"][u, at])):
                    x.append(y[ok])
            if st["lens"] is not None:
                m = int(st["lens"][b])
                at = st["block_table"][b, :-(-m // S)].long()
                for x, y in zip((k, v), _exact_record(st["cache"][at, h])):
                    x.append(y.reshape(-1, D)[:m])
            old = sum(x.shape[0] for x in k)
            k, v = torch.cat(k + [st["k"][b, :n, h].double()]), torch.cat(v + [st["v"][b, :n, h].double()])
            for j in range(h * g, h * g + g):
                s = (st["q"][b, :n, j].double() @ k.T) * st["scale"]
                s[:, old:].masked_fill_(~sees, -math.inf)
                out[b, :n, j] = torch.softmax(s, -1) @ v
    return {"o": out}


def _exact_verify(st):
    """A sequence at a time, with the rest of the probabilities renormalised after every refusal."""
    c = st["case"]
    B, T = c["batch"], c["nodes"]
    path = torch.full((B, T), -1, dtype=torch.int32)
    length, following = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    counts = st["counts"].tolist()
    parents, tokens = st["parents"].tolist(), st["tokens"].tolist()
    uniform = st["uniform"].double().tolist() if st["uniform"] is not None else None
    for b in range(B):
        at, walk = 0, [0]
        while True:
            full = st["target"][b, at].double()
            q = st["draft"][b, at].double() if st["draft"] is not None else None
            rest, total, found = full.clone(), 1.0, None
            for t in range(at + 1, counts[b]):
                if parents[b][t] != at:
                    continue
                x = tokens[b][t]
                if uniform is None:
                    ok = int((full == full.max()).nonzero()[0, 0]) == x
                elif q is None:
                    ok = uniform[b][t] * total < float(rest[x])
                    if not ok:
                        total = max(total - float(rest[x]), 0.0)
                        rest[x] = 0
                else:
                    ok = uniform[b][t] * float(q[x]) < float(rest[x])
                    if not ok:
                        rest = torch.clamp(rest - q, min=0)
                        rest = rest / rest.sum()
                if ok:
                    found = t
                    break
            if found is None:
                break
            walk.append(found)
            at = found
        if uniform is None:
            following[b] = int((full == full.max()).nonzero()[0, 0])
        else:
            if not float(rest.sum()) > 0:
                rest = full
            run = torch.cumsum(rest, 0)
            following[b] = int(torch.searchsorted(run, uniform[b][0] * run[-1:], right=True)[0])
        path[b, :len(walk)] = torch.tensor(walk, dtype=torch.int32)
        length[b] = len(walk)
    return {"path": path.to("cuda"), "n": length.to("cuda"), "next": following.to("cuda")}


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "verify":
        return _exact_verify(st)
    if c["op"] != "commit":
        return _exact_tree(st)
    out = {f: torch.zeros(st[f].shape, dtype=torch.float64, device="cuda") for f in ("k", "v")}
    for b, n in enumerate(st["n_path"].tolist()):
        for f in out:
            out[f][:, b, :n] = _exact_held(st[f][:, b, st["path"][b, :n].long()].double())
    return out
