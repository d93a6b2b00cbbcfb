"""Plain 64-bit restatement of the 4-bit pages, the rotation and the attention over them, from the formulas in
include/ice.h (torch on any device; shares no code with the library)."""
import math

import torch

D, S, G, RECORD = 128, 16, 64, 2304


def groups(x):
    """(step, mid) [..., 2, 2] in fp32 and codes [..., 128] (int64) of rows x [..., 128] (bf16 or fp32)."""
    g = x.double().unflatten(-1, (2, G))
    lo, hi = g.amin(-1), g.amax(-1)
    step = ((hi - lo) / 15).float().bfloat16()
    mid = ((hi + lo) / 2).float().bfloat16()
    bad = ~torch.isfinite((g.amax(-1).float() - g.amin(-1).float())) | torch.isnan(g).any(-1)
    step = torch.where(bad, torch.zeros_like(step), step)
    mid = torch.where(bad, torch.full_like(mid, math.nan), mid)
    st, mi = torch.where(step > 0, step, torch.ones_like(step)).double()[..., None], mid.double()[..., None]
    # x - mid with its rounding error (Knuth 1969): a tiny x beside a large mid is not lost; m * step is exact
    d = g - mi
    e = (g - (d - (d - g))) - (mi + (d - g))
    m = torch.round(torch.nan_to_num(d / st))
    rem = (d - m * st) + e
    even = m + 7 + (m.long() + 7) % 2  # the even one of m + 7 and m + 8
    c = torch.where(rem > 0, m + 8, torch.where(rem < 0, m + 7, even)).clamp(0, 15)
    c = torch.where((step > 0)[..., None], c, torch.zeros_like(c))
    return torch.stack((step, mid), -1), c.flatten(-2).long()


def values(meta, codes):
    m = meta.double()
    c = codes.double().unflatten(-1, (2, G))
    return (m[..., 1:2] + m[..., 0:1] * (c - 7.5)).flatten(-2)


def held(x):
    """What 4 bits hold of rows, in 64 bits."""
    return values(*groups(x))


def places(device):
    """Byte of every element's code in a record: K [16, 128] and V [16, 128] (low nibble for even elements)."""
    e = torch.arange(D, device=device)
    t = torch.arange(S, device=device)[:, None]
    w = e // 8
    k = 64 * t + 4 * (4 * (w % 4) + w // 4) + (e % 8) // 2
    p = e // 4
    v = 1152 + 4 * ((t // 2) * 32 + (p % 8) * 4 + p // 8) + 2 * (t % 2) + (e % 4) // 2
    return k, v


def encode(k, v):
    """Records [n, 2304] of rows [n, 16, 128]."""
    n = k.shape[0]
    out = torch.zeros((n, RECORD), dtype=torch.uint8, device=k.device)
    for x, at, off in zip((k, v), places(k.device), (1024, 2176)):
        meta, codes = groups(x)
        out[:, at[:, 0::2].reshape(-1)] = (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8).reshape(n, -1)
        out[:, off:off + 128] = meta.reshape(n, S * 4).contiguous().view(torch.uint8).view(n, 128)
    return out


def decode(rec):
    """K and V [n, 16, 128] in 64 bits."""
    n = rec.shape[0]
    got = []
    for at, off in zip(places(rec.device), (1024, 2176)):
        b = rec[:, at.reshape(-1)].view(n, S, D).long()
        codes = (b >> (4 * (torch.arange(D, device=rec.device) % 2))) & 15
        meta = rec[:, off:off + 128].contiguous().view(torch.bfloat16).view(n, S, 2, 2)
        got.append(values(meta, codes))
    return got


def norm(x, w, eps):
    x = x.double()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def rotate(x, cs, interleaved):
    """x [..., H, 128] in 64 bits, cs [..., rd / 2, 2] of each token."""
    cs = cs.double()[..., None, :, :]
    c, s = cs[..., 0], cs[..., 1]
    rd = 2 * c.shape[-1]
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rd:]), -1)


def attention(q, k, v, scale):
    """q [g, 128], k and v [n, 128] (64 bits): (O [g, 128], lse [g])."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=q.dtype, device=q.device)
    s = q @ k.T * scale
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]) @ v, lse


def attention_tolerance(q, k, v, scale):
    """Bounds on |O - O64| and |lse - lse64| of an fp32 attention.  A score is a sum of d = 128 products and of the
    two groups' (step, mid) terms: each partial sum is rounded by at most 2^-23 (a truncating adder counts a whole
    step) of the sum of absolute terms A = scale * (sum |q| |k - mid| + |q| |mid| and the code offset, at most 3 sum
    |q| |k|max); 16 roundings in sequence cover the 8-wide products (128 / 16), the groups and the scaling.  So a score is off
    by e = 16 * 2^-23 * 3 A, a weight exp(s) / sum by 2 e + 2^-20 (the exponential, the running maximum and the sums
    over pages), and O by that times max |v|, plus the weights' 22 bits (2^-21 max |v|, offsets of a code included)."""
    if k.shape[0] == 0:
        return 0.0, 0.0
    big = scale * float((q.abs() @ k.abs().amax(0)).max())
    e = 16 * 2.0 ** -23 * 3 * big
    return (2 * e + 2.0 ** -20 + 2.0 ** -21) * float(v.abs().max()) * 1.0, e + 2.0 ** -20 + 2.0 ** -22 * (big + 20)


def attention_rms_tolerance(q, k, v, scale):
    """Bounds on the norm of O - O64 of each head, for roundings that are independent of one another (four times what
    they leave; the norm covers 128 elements).  A score is made of products in units of a code, q (k - lo) with lo the
    group's lowest value, and of lo sum q, in at most 16 sums one after another, each off by up to 2^-24 of a partial sum
    of random signs (its root mean square: A); the queries' 22 bits add 2^-23 of a product.  With O = sum w v / sum w the
    derivative of O by a score is w (v - O): a score that is off by e moves O by w e |v - O|.  A weight's own 2^-21
    (exponential, 22 bits beside the step) moves it by up to w 2^-21 (|v| + |O|).  Sums of fp32 values leave 2^-20 of O."""
    if k.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=q.dtype, device=q.device)
    kg, qg = k.unflatten(-1, (2, G)), q.unflatten(-1, (2, G))
    lo = kg.amin(-1)
    spread = (kg - lo[..., None]).flatten(-2)
    A = (q.square() @ spread.square().T).sqrt() + (qg.sum(-1)[:, None] * lo[None]).abs().sum(-1)
    e = scale * (4 * 2.0 ** -24 * A + 2.0 ** -23 * (q.square() @ k.square().T).sqrt())
    w = torch.softmax(q @ k.T * scale, -1)
    o = w @ v
    size = v.norm(dim=-1) + o.norm(dim=-1, keepdim=True)
    away = (v.square().sum(-1) - 2 * (o @ v.T) + o.square().sum(-1, keepdim=True)).clamp(min=0).sqrt()
    return 4 * (w * (e * away + 2.0 ** -21 * size)).square().sum(-1).sqrt() + 2.0 ** -20 * o.norm(dim=-1)
