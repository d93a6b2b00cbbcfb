"""The 64-bit restatement of the 4-bit pages that the GPU tests compare with: its layout against include/ice.h's
words on hand-made rows, and its quantiser's error."""
import torch

import cache4_ref as ref


def test_layout_by_hand():
    k, v = torch.zeros((1, 16, 128)), torch.zeros((1, 16, 128))
    # group 0 of token 3: -7.5 .. 7.5 step 1 four times -> codes 0 .. 15; group 1 constant
    ramp = torch.arange(16).float() - 7.5
    k[0, 3, :64], k[0, 3, 64:] = ramp.repeat(4), 2.0
    v[0, 5, 64:] = ramp.repeat(4)
    r = ref.encode(k, v)[0]
    # elements 8 w ..: word 4 (w % 4) + w / 4 of the token's 64 bytes, low nibble first
    for w in range(8):
        at = 64 * 3 + 4 * (4 * (w % 4) + w // 4)
        want = [0x10, 0x32, 0x54, 0x76] if w % 2 == 0 else [0x98, 0xBA, 0xDC, 0xFE]
        assert r[at:at + 4].tolist() == want
    assert r[1024 + 24:1024 + 32].view(torch.bfloat16).tolist() == [1.0, 0.0, 0.0, 2.0]
    # V elements 4 p .. of token 5: the high half of word (2 * 8 + p % 8) * 4 + p / 8
    for p in range(16, 32):
        at = 1152 + 4 * ((2 * 8 + p % 8) * 4 + p // 8) + 2
        assert r[at:at + 2].tolist() == [[0x10, 0x32], [0x54, 0x76], [0x98, 0xBA], [0xDC, 0xFE]][p % 4]
    K, V = ref.decode(r[None])
    assert torch.equal(K, k.double()) and torch.equal(V, v.double())


def test_every_byte_once():
    k, v = ref.places("cpu")
    at = torch.cat((k[:, 0::2].flatten(), v[:, 0::2].flatten()))
    assert at.unique().numel() == 2048 and torch.equal(k[:, 0::2], k[:, 1::2]) and torch.equal(v[:, 0::2], v[:, 1::2])
    assert not bool(((at >= 1024) & (at < 1152)).any()) and int(at.max()) < 2176


def test_quantiser_error():
    x = torch.randn((200, 128), generator=torch.Generator().manual_seed(0)) * 3 + 1
    for t in (torch.float32, torch.bfloat16):
        y = x.to(t)
        meta, _ = ref.groups(y)
        step, mid = meta[..., 0].double(), meta[..., 1].double()
        # half a step, and what the rounding of step (7.5 steps) and mid leave outside the codes' range
        tol = step * (0.5 + 7.5 * 2.0 ** -8) + mid.abs() * 2.0 ** -8
        assert bool(((ref.held(y) - y.double()).abs().unflatten(-1, (2, 64)).amax(-1) <= tol).all())


def test_held_again_is_the_same():
    x = torch.randn((50, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    m1, c1 = ref.groups(x)
    assert int(c1.max()) == 15 and int(c1.min()) == 0 and m1.dtype == torch.bfloat16
