"""Refusals of the entry points for trees of drafted tokens, as include/ice.h states them: one broken argument each,
answered on the host before anything is launched.  Host addresses stand in for device pointers, so the file runs only
where no CUDA device is present."""
import ctypes

import numpy as np
import pytest
import torch

import semantic_paged_kv_gb300 as ice

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses stand in for device pointers")

_BUF = np.zeros(1 << 16, np.uint8)
A = (_BUF.ctypes.data + 255) & ~255
INV, UNS = ice.ICE_ERR_INVALID_ARG, ice.ICE_ERR_UNSUPPORTED
BIG = 1 << 40


def _p(**kw):
    p = ice.Config(batch=2, n_q_heads=8, n_kv_heads=2, n_tokens=100).params()
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _with(x, **kw):
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def _rows(**kw):
    return _with(ice.IceRows(A, 8192, 1024, 128), **kw)


def _tree(**kw):
    return _with(ice.IceTree(A, A, 5), **kw)


def _cache(**kw):
    return _with(ice.IceCache4(A, A, 10, 5), **kw)


def _probs(**kw):
    return _with(ice.IceProbs(A, 500, 100), **kw)


def _ref(x):
    return None if x is None else ctypes.byref(x)


OK = object()


def _or(x, make):
    return _ref(make() if x is OK else x)


def _attn(p=OK, tree=OK, q=OK, cache=OK, lens=A, k=OK, v=OK, scale=0.1, O=OK, ws=A, ws_bytes=BIG):
    return ice.load().ice_cache4_attn_tree(_or(p, _p), _or(tree, _tree), _or(q, _rows), _or(cache, _cache), lens,
                                           _or(k, _rows), _or(v, _rows), scale, _or(O, _rows), ws, ws_bytes, None, None)


def _sparse(p=OK, tree=OK, rec=A, page_len=A, sel=A, count=A, max_sel=4, cache=OK, lens=A, O=OK, ws=A):
    return ice.load().ice_sparse_attn_tree4(_or(p, _p), _or(tree, _tree), _ref(_rows()), rec, page_len, sel, count,
                                            max_sel, _or(cache, _cache), lens, _ref(_rows()), _ref(_rows()), 0.1,
                                            _or(O, _rows), ws, BIG, None, None)


def _verify(batch=2, vocab=100, dtype=ice.ICE_FP32, tree=OK, target=OK, draft=OK, tokens=A, uniform=A, path=A, n=A,
            nxt=A):
    return ice.load().ice_tree_verify(batch, vocab, dtype, _or(tree, _tree), _or(target, _probs), _or(draft, _probs),
                                      tokens, uniform, path, n, nxt, None, None)


def _commit(p=OK, layers=2, nodes=5, k=OK, v=OK, kl=4096, vl=4096, path=A, n=A, start=A, cache=OK, rl=10 * 2 * 2304):
    return ice.load().ice_cache4_commit(_or(p, _p), layers, nodes, _or(k, _rows), _or(v, _rows), kl, vl, path, n, start,
                                        _or(cache, _cache), rl, None, None)


REFUSED = [
    (lambda: _attn(p=None), INV), (lambda: _attn(p=_p(head_dim=64)), UNS), (lambda: _attn(tree=None), INV),
    (lambda: _attn(tree=_tree(n_nodes=-1)), INV), (lambda: _attn(tree=_tree(n_nodes=257)), UNS),
    (lambda: _attn(q=None), INV), (lambda: _attn(q=_rows(data=A + 8)), INV), (lambda: _attn(q=_rows(token=1025)), INV),
    (lambda: _attn(k=None), INV), (lambda: _attn(k=_rows(head=-128)), INV), (lambda: _attn(v=_rows(data=None)), INV),
    (lambda: _attn(O=_rows(head=64)), INV), (lambda: _attn(O=None), INV), (lambda: _attn(cache=None), INV),
    (lambda: _attn(lens=None), INV), (lambda: _attn(cache=_cache(n_pages=0)), INV),
    (lambda: _attn(cache=_cache(records=A + 8)), INV), (lambda: _attn(scale=float("nan")), INV),
    (lambda: _attn(scale=float("inf")), INV), (lambda: _attn(ws=None), INV), (lambda: _attn(ws=A + 16), INV),
    (lambda: _attn(tree=_tree(parents=None, n_nodes=1 << 30)), UNS), (lambda: _attn(ws_bytes=1000), INV),
    (lambda: _sparse(rec=None), INV), (lambda: _sparse(rec=A + 4), INV), (lambda: _sparse(page_len=None), INV),
    (lambda: _sparse(sel=None), INV), (lambda: _sparse(count=None), INV), (lambda: _sparse(max_sel=0), INV),
    (lambda: _sparse(max_sel=1 << 27), UNS), (lambda: _sparse(cache=None), INV), (lambda: _sparse(lens=None), INV),
    (lambda: _sparse(tree=None), INV), (lambda: _sparse(O=None), INV),
    (lambda: _verify(batch=0), INV), (lambda: _verify(vocab=0), INV), (lambda: _verify(dtype=2), INV),
    (lambda: _verify(vocab=(1 << 28) + 1), UNS), (lambda: _verify(batch=1 << 24), UNS),
    (lambda: _verify(tree=None), INV), (lambda: _verify(tree=_tree(n_nodes=0)), INV),
    (lambda: _verify(tree=_tree(n_nodes=1025)), UNS), (lambda: _verify(target=None), INV),
    (lambda: _verify(target=_probs(data=A + 2)), INV), (lambda: _verify(target=_probs(batch=-1)), INV),
    (lambda: _verify(draft=_probs(data=None)), INV), (lambda: _verify(draft=_probs(node=-5)), INV),
    (lambda: _verify(tokens=None), INV), (lambda: _verify(path=None), INV), (lambda: _verify(n=None), INV),
    (lambda: _verify(nxt=None), INV),
    (lambda: _commit(p=None), INV), (lambda: _commit(layers=-1), INV), (lambda: _commit(layers=1 << 30), UNS),
    (lambda: _commit(nodes=-1), INV), (lambda: _commit(k=None), INV), (lambda: _commit(v=_rows(data=A + 4)), INV),
    (lambda: _commit(kl=4), INV), (lambda: _commit(vl=-8), INV), (lambda: _commit(rl=8), INV),
    (lambda: _commit(rl=10 * 2 * 2304 - 16), INV), (lambda: _commit(path=None), INV), (lambda: _commit(n=None), INV),
    (lambda: _commit(start=None), INV), (lambda: _commit(cache=None), INV),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(i):
    call, status = REFUSED[i]
    assert call() == status
    assert ice.load().ice_last_error()


def test_nothing_to_do():
    """Calls of no node or layer answer without a launch."""
    assert _attn(tree=_tree(n_nodes=0)) == ice.ICE_OK
    assert _attn(tree=_tree(parents=None, n_nodes=0)) == ice.ICE_OK
    assert _sparse(tree=_tree(n_nodes=0)) == ice.ICE_OK
    assert _commit(nodes=0) == ice.ICE_OK and _commit(layers=0) == ice.ICE_OK


def test_workspace_bytes():
    n = ctypes.c_size_t(0)
    assert ice.load().ice_tree_workspace_bytes(ctypes.byref(_p()), None) == INV
    assert ice.load().ice_tree_workspace_bytes(ctypes.byref(_p()), ctypes.byref(n)) == ice.ICE_OK and n.value > 0


def test_binding_checks():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in (lambda: ice.Tree(i32(2, 5).long()), lambda: ice.Tree(i32(2, 5), n_nodes=4), lambda: ice.Tree(i32(5)),
                lambda: ice.Tree(None), lambda: ice.Tree(i32(2, 5), i32(2, 1)), lambda: ice.Tree(i32(4, 5)[::2].t()),
                lambda: ice.probs(torch.zeros(2, 5)), lambda: ice.probs(torch.zeros(2, 5, 7).half()),
                lambda: ice.probs(torch.zeros(2, 7, 5).transpose(1, 2))):
        with pytest.raises(ice.IceError) as e:
            bad()
        assert e.value.status == INV
    t, pr = ice.Tree(i32(2, 5)), ice.probs(torch.zeros(2, 5, 7))
    ok = dict(tokens=i32(2, 5), uniform=torch.zeros(2, 5), path=i32(2, 5), n_path=i32(2), next_token=i32(2))
    for f, x in (("tokens", i32(2, 4)), ("uniform", torch.zeros(2, 5).double()), ("path", i32(2, 10)[:, ::2]),
                 ("n_path", i32(3)), ("next_token", i32(2).long())):
        with pytest.raises(ice.IceError):
            ice.ice_tree_verify(t, pr, pr, **{**ok, f: x}, err=None, stream=0)
    with pytest.raises(ice.IceError):
        ice.ice_tree_verify(ice.Tree(i32(2, 6)), pr, pr, **ok, err=None, stream=0)
    with pytest.raises(ice.IceError):
        ice.ice_tree_verify(t, pr, ice.probs(torch.zeros(2, 5, 8)), **ok, err=None, stream=0)


def test_too_much_work():
    """More tiles than a run can count; the same nodes behind fewer pages are not refused for it."""
    tree = lambda: _tree(parents=None, n_nodes=1 << 20)  # noqa: E731
    assert _attn(tree=tree(), cache=_cache(max_pages=1 << 26)) == UNS
    assert "too much work" in ice.load().ice_last_error().decode()
    assert _attn(tree=tree(), cache=_cache(max_pages=1 << 16), ws_bytes=1000) == INV
    assert _sparse(tree=tree(), max_sel=1 << 26) == UNS
    assert "too much work" in ice.load().ice_last_error().decode()


def test_binding_checks_the_batch_of_a_tree():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pr = ice.probs(torch.zeros(2, 5, 7))
    ok = dict(tokens=i32(2, 5), uniform=torch.zeros(2, 5), path=i32(2, 5), n_path=i32(2), next_token=i32(2))
    for t in (ice.Tree(i32(1, 5)), ice.Tree(i32(2, 5), i32(3)), ice.Tree(None, i32(1), 5)):
        with pytest.raises(ice.IceError) as e:
            ice.ice_tree_verify(t, pr, pr, **ok, err=None, stream=0)
        assert e.value.status == INV
        with pytest.raises(ice.IceError) as e:
            ice.ice_cache4_attn_tree(_p(), t, _rows(), None, None, _rows(), _rows(), 0.1, _rows(), None, None, stream=0)
        assert e.value.status == INV and "sequences" in str(e.value)
