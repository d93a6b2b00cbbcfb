"""The bound that the attention tests put on an error's norm: fp32 arithmetic keeps it, and it rejects weights or queries
of fewer bits, a page or a token left out, and a wrong weight in a join."""
import pytest
import torch

import cache4_ref as ref

SCALE = 0.088


def _case(n, seed=0, g=8):
    gen = torch.Generator().manual_seed(seed)
    k, v = (ref.held(torch.randn((n, 128), generator=gen).bfloat16()) for _ in range(2))
    q = torch.randn((g, 128), generator=gen)
    return q, k, v


def _over(O, q, k, v):
    o, _ = ref.attention(q.double(), k, v, SCALE)
    return (O.double() - o).norm(dim=-1) / ref.attention_rms_tolerance(q.double(), k, v, SCALE)


def _weights(q, k):
    return torch.softmax(q.double() @ k.T * SCALE, -1)


@pytest.mark.parametrize("n", [1, 17, 1000, 40000])
def test_fp32_is_within(n):
    q, k, v = _case(n)
    s = q @ k.float().T * SCALE
    p = torch.exp(s - s.amax(-1, keepdim=True))
    O = p @ v.float() / p.sum(-1, keepdim=True)
    assert float(_over(O, q, k, v).max()) < 1


@pytest.mark.parametrize("n", [100, 4097, 40000])
def test_fewer_bits_and_missing_parts_are_not(n):
    q, k, v = _case(n, 1)
    w = _weights(q, k)
    bad = {"bf16 weights": w.bfloat16().double() @ v, "fp16 weights": (w * n).half().double() @ v / n,
           "fp16 queries": ref.attention(q.half().double(), k, v, SCALE)[0],
           "a page's values": w @ torch.where(torch.arange(n)[:, None] // 16 == 3, 0.0, v),
           "a token": ref.attention(q.double(), torch.cat((k[:50], k[51:])), torch.cat((v[:50], v[51:])), SCALE)[0],
           "the second of two tokens swapped": w @ torch.cat((v[:20], v[21:22], v[20:21], v[22:]))}
    half = torch.where(torch.arange(n) < n // 2, 1.01, 1.0).double()
    bad["a join's weight"] = (w * half) @ v / (w * half).sum(-1, keepdim=True)
    for what, O in bad.items():
        assert float(_over(O, q, k, v).min()) > 1, what
