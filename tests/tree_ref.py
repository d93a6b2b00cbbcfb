"""Plain 64-bit restatement of the attention of drafted trees and of their verification, from the formulas in
include/ice.h (torch on any device; shares no code with the library)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of the storage type, relative


def sees(parents, n, device="cpu"):
    """[n, n]: whether node i attends to node j (parents: a list, or None for a chain)."""
    m = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        up = i - 1 if parents is None else parents[i]
        if up >= 0:
            m[i] = m[up]
        m[i, i] = True
    return m.to(device)


def attention(q, k, v, keep, scale):
    """q [T, 128], k and v [n, 128], keep [T, n] in 64 bits: O [T, 128]; masked values take no part."""
    s = (q @ k.T * scale).masked_fill(~keep, -math.inf)
    w = torch.softmax(s, -1)
    if bool(torch.isfinite(v).all()):
        return w @ v
    out = torch.empty((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
    for i in range(q.shape[0]):
        out[i] = w[i, keep[i]] @ v[keep[i]]
    return out


def tolerance(q, k, v, keep, scale, dtype):
    """Bounds on |O - O64| (norms of rows of 128 elements) for roundings that are independent of one another, four times
    what they leave.
    bf16: keys, values and weights go in as fp16 numbers, off by up to half a step, 2^-11 of themselves.  A score, a sum
    of products q k whose k is rounded so, is off by about e = scale 2^-11 sqrt(sum q^2 k^2); with O = sum w v / sum w
    the derivative of O by a score is w (v - O), so it moves O by w e |v - O|; a weight's and a value's own rounding move
    it by w 2^-11 |v| each.  fp32: e = scale 2^-24 16 sqrt(sum q^2 k^2) (sums of 128 products, rounded up to 128 times
    with partial sums of random signs) and the score's own rounding, 2^-22 |s|; weights 2^-21.
    Sums of thousands of terms: 2^-18 of O, fp32 2^-20 (partial sums of random signs, joined over runs); then O is rounded once."""
    w = torch.softmax((q @ k.T * scale).masked_fill(~keep, -math.inf), -1)
    o = w @ v
    fine, step = (2.0 ** -11, 2 * 2.0 ** -11) if dtype == torch.bfloat16 else (16 * 2.0 ** -24, 2.0 ** -21)
    e = scale * fine * (q.square() @ k.square().T).sqrt() + 2.0 ** -22 * (q @ k.T * scale).abs()
    away = (v.square().sum(-1) - 2 * (o @ v.T) + o.square().sum(-1, keepdim=True)).clamp(min=0).sqrt()
    err = 4 * (w * (e * away + step * v.norm(dim=-1))).square().sum(-1).sqrt()
    return err + ((2.0 ** -18 if dtype == torch.bfloat16 else 2.0 ** -20) + HALF[dtype]) * o.norm(dim=-1)


def verify(target, draft, tokens, parents, uniform, n):
    """One sequence: target and draft [T, V] in 64 bits, tokens, parents (None: a chain) and uniform as lists.  Returns
    (path, next token), and how near the nearest decision came to its border (relative)."""
    vocab = target.shape[1]
    if n == 0:
        return [], -1, 1.0
    clean = lambda x: torch.where(x > 0, x, torch.zeros_like(x))  # noqa: E731  (NaN and negative: 0)
    path, at, near = [0], 0, 1.0
    while True:
        p = target[at]
        q = draft[at] if draft is not None else None
        beta, mass, left, found = 0.0, 1.0, p.clone(), None
        for c in range(at + 1, n):
            if (c - 1 if parents is None else parents[c]) != at or not 0 <= tokens[c] < vocab:
                continue
            x = tokens[c]
            if uniform is None:
                ok = x == largest(p)
            elif q is None:
                a, b = uniform[c] * mass, float(left[x])
                ok = a < b
                near = min(near, abs(a - b) / max(a, b, 1e-300))
                if not ok and b > 0:
                    mass, left[x] = max(mass - b, 0.0), 0.0
            else:
                a, b = uniform[c] * float(q[x]) * mass, float(p[x]) - beta * float(q[x])
                ok = a < b
                if a or b:
                    near = min(near, abs(a - b) / max(abs(a), abs(b), 1e-300))
                if not ok and mass > 0:
                    beta += mass
                    mass = float(clean(p - beta * q).sum())
            if ok:
                found = c
                break
        if found is None:
            break
        path.append(found)
        at = found
    if uniform is None:
        return path, largest(p), 1.0
    w = clean(left if q is None else p - beta * q)
    if not float(w.sum()) > 0:
        w = clean(p)
    run = w.cumsum(0)
    total = float(run[-1])
    if not total > 0:
        return path, -1, near
    want = uniform[0] * total
    hit = (run > want).nonzero()
    nxt = int(hit[0, 0]) if len(hit) else int((w > 0).nonzero()[-1, 0])
    gaps = (run - want).abs()
    if want > 0:
        near = min(near, float(gaps.min()) / total)
    return path, nxt, near


def largest(p):
    p = torch.where(torch.isnan(p), torch.full_like(p, -math.inf), p)
    if not bool((p > -math.inf).any()):
        return -1
    return int((p == p.max()).nonzero()[0, 0])
