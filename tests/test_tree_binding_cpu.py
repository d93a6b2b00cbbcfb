"""What the binding checks of the tensors of a call for drafted trees, before anything is launched (CPU tensors: every call
here is refused, or has nothing to do)."""
import pytest
import torch

import semantic_paged_kv_gb300 as ice

B, T, HQ, HKV, CAP, SEL = 2, 5, 8, 2, 7, 4
I32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731


def _params(**kw):
    return ice.Config(batch=B, n_q_heads=HQ, n_kv_heads=HKV, n_tokens=0, np_cap=1, page_cap=CAP, **kw).params()


def _rows(heads, n=T, batch=B, dtype=torch.bfloat16):
    return ice.rows(torch.zeros((batch, n, heads, 128), dtype=dtype))


def _cache(heads=HKV, batch=B):
    return ice.Cache4(torch.zeros((10, heads, 2304), dtype=torch.uint8), I32(batch, 3))


def _attn(**kw):
    a = dict(tree=ice.Tree(I32(B, T)), q=_rows(HQ), cache=_cache(), lens=I32(B), k=_rows(HKV), v=_rows(HKV), O=_rows(HQ))
    a.update(kw)
    ice.ice_cache4_attn_tree(_params(), a["tree"], a["q"], a["cache"], a["lens"], a["k"], a["v"], 0.1, a["O"], None, None,
                             stream=0)


def _sparse(**kw):
    U = B * HKV
    a = dict(q=_rows(HQ), page_len=I32(U, CAP), sel_pages=I32(U, SEL), sel_count=I32(U), cache=_cache(), lens=I32(B),
             k=_rows(HKV), v=_rows(HKV), O=_rows(HQ))
    a.update(kw)
    ice.ice_sparse_attn_tree4(_params(), ice.Tree(I32(B, T)), a["q"], torch.zeros((U, CAP, 2304), dtype=torch.uint8),
                              a["page_len"], a["sel_pages"], a["sel_count"], a["cache"], a["lens"], a["k"], a["v"], 0.1,
                              a["O"], None, None, stream=0)


def _commit(**kw):
    a = dict(k=_rows(HKV), v=_rows(HKV), path=I32(B, T), n_path=I32(B), start=I32(B), cache=_cache(), layers=1)
    a.update(kw)
    ice.ice_cache4_commit(_params(), a["layers"], T, a["k"], a["v"], a["path"], a["n_path"], a["start"], a["cache"], None,
                          stream=0)


SPACED = torch.zeros(2 * B, dtype=torch.int32)[::2]
REFUSED = [
    (_attn, "lens", I32(B).long()), (_attn, "lens", I32(B - 1)), (_attn, "lens", SPACED), (_attn, "lens", I32(B).float()),
    (_attn, "q", _rows(HQ, T - 1)), (_attn, "q", _rows(HQ - 1)), (_attn, "k", _rows(HKV, 2)), (_attn, "v", _rows(HKV, T - 1)),
    (_attn, "O", _rows(HQ, batch=1)), (_attn, "O", _rows(HQ, dtype=torch.float32)),
    (_attn, "cache", _cache(heads=1)), (_attn, "cache", _cache(batch=1)),
    (_sparse, "lens", I32(B).long()), (_sparse, "page_len", I32(B * HKV, CAP - 1)), (_sparse, "page_len", I32(B * HKV)),
    (_sparse, "sel_pages", I32(B * HKV, SEL).long()), (_sparse, "sel_pages", I32(B * HKV - 1, SEL)),
    (_sparse, "sel_pages", I32(SEL, B * HKV).t()), (_sparse, "sel_count", I32(B * HKV).long()),
    (_sparse, "sel_count", I32(B)), (_sparse, "q", _rows(HQ, dtype=torch.float32)),
    (_commit, "path", I32(B, T).long()), (_commit, "path", I32(B, T + 1)), (_commit, "path", I32(B, 2 * T)[:, ::2]),
    (_commit, "n_path", I32(B).long()), (_commit, "n_path", I32(1)), (_commit, "start", I32(B).long()),
    (_commit, "start", SPACED), (_commit, "k", _rows(HKV, T - 1)), (_commit, "v", _rows(HKV, dtype=torch.float32)),
    (_commit, "cache", _cache(heads=3)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(i):
    call, name, x = REFUSED[i]
    with pytest.raises(ice.IceError) as e:
        call(**{name: x})
    assert e.value.status == ice.ICE_ERR_INVALID_ARG
    assert name in str(e.value)


def test_what_is_larger_than_needed_passes():
    """Tensors made for a larger batch or more nodes, and rows that are the same for all, come as far as the library's own
    checks."""
    for call, kw in ((_attn, dict(lens=I32(B + 3), q=_rows(HQ, T + 1, B + 1), cache=_cache(batch=B + 1))),
                     (_attn, dict(k=_rows(HKV, batch=1), v=_rows(1), q=_rows(HQ, 1))),
                     (_sparse, dict(sel_count=I32(3 * B * HKV), sel_pages=I32(B, HKV, SEL)))):
        with pytest.raises(ice.IceError) as e:
            call(**kw)
        assert "workspace" in str(e.value)
    _commit(n_path=I32(B + 1), start=I32(B + 1), path=I32(B + 1, T), layers=0)
