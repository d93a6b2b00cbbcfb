"""Refusals of the rotation, 4-bit cache and 4-bit pool entry points, as include/ice.h states them: one broken
argument each, answered on the host before anything is launched.  Host addresses stand in for device pointers, so the
file runs only where no CUDA device is present."""
import ctypes

import numpy as np
import pytest
import torch

import semantic_paged_kv_gb300 as ice

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses stand in for device pointers")

_BUF = np.zeros(1 << 16, np.uint8)
A = (_BUF.ctypes.data + 255) & ~255
INV, UNS = ice.ICE_ERR_INVALID_ARG, ice.ICE_ERR_UNSUPPORTED


def _p(**kw):
    p = ice.Config(batch=2, n_q_heads=8, n_kv_heads=2, n_tokens=100).params()
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _rows(**kw):
    r = ice.IceRows(A, 1024, 256, 128)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _rope(**kw):
    r = ice.IceRope(A, 100, 128, 0, 1e-6, None, None)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _cache(**kw):
    c = ice.IceCache4(A, A, 10, 5)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _ref(x):
    return None if x is None else ctypes.byref(x)


OK = object()


def _qkv(p=None, n=3, q=OK, k=OK, v=OK, rope=OK, qo=OK, ko=OK, vo=OK):
    d = lambda x: _ref(_rows() if x is OK else x)  # noqa: E731
    return ice.load().ice_qkv_rope(ctypes.byref(p or _p()), n, d(q), d(k), d(v), None, None, None,
                                   _ref(_rope() if rope is OK else rope), d(qo), d(ko), d(vo), None, None)


def _append(p=None, n=3, k=OK, q=None, qo=None, rope=None, start=A, cache=OK):
    return ice.load().ice_cache4_append(ctypes.byref(p or _p()), n, _ref(q), _ref(_rows() if k is OK else k),
                                        _ref(_rows()), None, start, None, _ref(rope), _ref(qo),
                                        _ref(_cache() if cache is OK else cache), None, None)


def _read(n=3, start=A, cache=OK, vo=OK):
    return ice.load().ice_cache4_read(ctypes.byref(_p()), n, _ref(_cache() if cache is OK else cache), start, None,
                                      _ref(_rows()), _ref(_rows() if vo is OK else vo), None, None)


def _index(**null):
    ix = ice.IceIndex(*[A] * len(ice.INDEX_FIELDS))
    for f, x in null.items():
        setattr(ix, f, x)
    return ix


def _pack(p=None, ix=OK, first=0, rec=A):
    return ice.load().ice_pool4_pack(ctypes.byref(p or _p()), _ref(_index() if ix is OK else ix), first, rec, None, None)


def _unpack(ix=OK, rec=A):
    return ice.load().ice_pool4_unpack(ctypes.byref(_p()), _ref(_index() if ix is OK else ix), rec, None, None)


def _attn(p=None, q=A, cache=OK, lens=A, o=A, lse=None, ws=A, n=1 << 40):
    return ice.load().ice_cache4_attn_decode(ctypes.byref(p or _p()), q, _ref(_cache() if cache is OK else cache), lens,
                                             0.1, o, lse, ws, n, None, None)


def _sparse(rec=A, pl=A, sel=A, cnt=A, most=4, cache=None, lens=None, ws=A, n=1 << 40):
    return ice.load().ice_sparse_attn_decode4(ctypes.byref(_p()), A, rec, pl, sel, cnt, most, _ref(cache), lens, 0.1, A,
                                              None, ws, n, None, None)


def _table(inv=A, rd=128, n=10, t=A):
    return ice.load().ice_rope_table(inv, rd, n, t, None)


CASES = [
    ("table: NULL", lambda: _table(inv=None), INV, "inv_freq"),
    ("table: misaligned", lambda: _table(t=A + 4), INV, "16-byte aligned"),
    ("table: odd rotary", lambda: _table(rd=40), UNS, "rotary_dim"),
    ("table: no position", lambda: _table(n=0), INV, "n_positions"),
    ("rope: head_dim", lambda: _qkv(p=_p(head_dim=64)), UNS, "head_dim"),
    ("rope: q without q_out", lambda: _qkv(qo=None), INV, "q_out is NULL"),
    ("rope: k_out without k", lambda: _qkv(k=None), INV, "k is NULL"),
    ("rope: NULL data", lambda: _qkv(v=_rows(data=None)), INV, "v must be"),
    ("rope: misaligned data", lambda: _qkv(ko=_rows(data=A + 8)), INV, "k_out must be"),
    ("rope: stride of 8 bytes", lambda: _qkv(q=_rows(token=132)), INV, "q: strides"),
    ("rope: negative stride", lambda: _qkv(q=_rows(head=-128)), INV, "q: strides"),
    ("rope: output rows on one another", lambda: _qkv(ko=_rows(head=0)), INV, "k_out: a stride below d"),
    ("read: output rows on one another", lambda: _read(vo=_rows(token=64)), INV, "v_out: a stride below d"),
    ("rope: rotary_dim too large", lambda: _qkv(rope=_rope(rotary_dim=144)), UNS, "rotary_dim"),
    ("rope: rotary_dim 0", lambda: _qkv(rope=_rope(rotary_dim=0)), UNS, "rotary_dim"),
    ("rope: interleaved 2", lambda: _qkv(rope=_rope(interleaved=2)), INV, "interleaved"),
    ("rope: no position", lambda: _qkv(rope=_rope(n_positions=0)), INV, "n_positions"),
    ("rope: table misaligned", lambda: _qkv(rope=_rope(table=A + 4)), INV, "table"),
    ("rope: weights misaligned", lambda: _qkv(rope=_rope(k_norm=A + 2)), INV, "k_norm"),
    ("rope: eps NaN", lambda: _qkv(rope=_rope(q_norm=A, eps=float("nan"))), INV, "eps"),
    ("rope: negative n_new", lambda: _qkv(n=-1), INV, "n_new"),
    ("rope: too many rows", lambda: _qkv(n=1 << 30), UNS, "too many rows"),
    ("append: k NULL", lambda: _append(k=None), INV, "k is NULL"),
    ("append: q without q_out", lambda: _append(q=_rows()), INV, "q_out is NULL"),
    ("append: start NULL", lambda: _append(start=None), INV, "start is NULL"),
    ("append: cache NULL", lambda: _append(cache=None), INV, "cache is NULL"),
    ("append: records misaligned", lambda: _append(cache=_cache(records=A + 8)), INV, "records"),
    ("append: block table NULL", lambda: _append(cache=_cache(table=None)), INV, "table is NULL"),
    ("append: no page", lambda: _append(cache=_cache(n_pages=0)), INV, "n_pages"),
    ("append: positions beyond int32", lambda: _append(cache=_cache(max_pages=1 << 27)), UNS, "max_pages"),
    ("read: start NULL", lambda: _read(start=None), INV, "start is NULL"),
    ("read: v_out misaligned", lambda: _read(vo=_rows(data=A + 2)), INV, "v_out"),
    ("read: cache NULL", lambda: _read(cache=None), INV, "cache is NULL"),
    ("pack: index NULL", lambda: _pack(ix=None), INV, "index is NULL"),
    ("pack: pool NULL", lambda: _pack(ix=_index(pool_v=None)), INV, "pool_k and pool_v"),
    ("pack: page_len NULL", lambda: _pack(ix=_index(page_len=None)), INV, "page_len"),
    ("pack: token_slot NULL", lambda: _pack(ix=_index(token_slot=None), first=5), INV, "token_slot"),
    ("pack: negative first token", lambda: _pack(first=-1), INV, "first_token"),
    ("pack: records misaligned", lambda: _pack(rec=A + 4), INV, "records"),
    ("pack: too many pages", lambda: _pack(p=_p(page_cap=1 << 30)), UNS, "too many pages"),
    ("unpack: records NULL", lambda: _unpack(rec=None), INV, "records"),
    ("unpack: n_pages NULL", lambda: _unpack(ix=_index(n_pages=None)), INV, "n_pages"),
    ("attention: Q NULL", lambda: _attn(q=None), INV, "non-NULL Q"),
    ("attention: O misaligned", lambda: _attn(o=A + 4), INV, "Q and O"),
    ("attention: lse misaligned", lambda: _attn(lse=A + 2), INV, "lse"),
    ("attention: lens NULL", lambda: _attn(lens=None), INV, "lens is NULL"),
    ("attention: cache NULL", lambda: _attn(cache=None), INV, "cache is NULL"),
    ("attention: workspace too small", lambda: _attn(n=16), INV, "workspace has"),
    ("attention: workspace misaligned", lambda: _attn(ws=A + 16), INV, "256-byte"),
    ("attention: 17 heads a group", lambda: _attn(p=_p(n_q_heads=34)), UNS, "16 query heads"),
    ("sparse: records NULL", lambda: _sparse(rec=None), INV, "records"),
    ("sparse: page_len NULL", lambda: _sparse(pl=None), INV, "page_len"),
    ("sparse: sel_count NULL", lambda: _sparse(cnt=None), INV, "sel_count"),
    ("sparse: max_sel 0", lambda: _sparse(most=0), INV, "max_sel"),
    ("sparse: cache without lens", lambda: _sparse(cache=_cache()), INV, "lens"),
    ("sparse: lens without cache", lambda: _sparse(lens=A), INV, "lens"),
]


@pytest.mark.parametrize("call,status,message", [pytest.param(*c[1:], id=c[0]) for c in CASES])
def test_refusal(call, status, message):
    assert call() == status
    assert message in ice.load().ice_last_error().decode()


def test_nothing_to_do_is_ok():
    assert _qkv(n=0, q=_rows(token=0), qo=_rows(token=0)) == ice.ICE_OK  # no second token to lie on the first
    assert _qkv(n=0) == ice.ICE_OK and _append(n=0) == ice.ICE_OK and _read(n=0) == ice.ICE_OK
    assert _qkv(q=None, qo=None, k=None, ko=None, v=None, vo=None) == ice.ICE_OK


@pytest.mark.parametrize("call", [
    lambda: ice.rows(torch.zeros(2, 3, 4, 64)), lambda: ice.rows(torch.zeros(2, 3, 128)),
    lambda: ice.rows(torch.zeros(2, 3, 128, 4).transpose(2, 3)),
    lambda: ice.Rope(torch.zeros(5, 64, 2, dtype=torch.float64)), lambda: ice.Rope(q_norm=torch.zeros(64)),
    lambda: ice.Cache4(torch.zeros(2, 2, 2304), torch.zeros(2, 2, dtype=torch.int32)),
    lambda: ice.Cache4(torch.zeros(2, 2, 2304, dtype=torch.uint8), torch.zeros(2, 2)),
    lambda: ice.ice_rope_table(torch.zeros(64), 5, torch.zeros(5, 64, 2)),
    lambda: ice.ice_rope_table(torch.zeros(64).double(), 6, torch.zeros(5, 64, 2))])
def test_binding_refusals(call):
    with pytest.raises(ice.IceError) as e:
        call()
    assert e.value.status == INV


def test_rows_strides():
    t = torch.zeros(2, 5, 12, 128)
    r = ice.rows(t[:, :, 8:10])
    assert (r.batch, r.token, r.head) == (5 * 12 * 128, 12 * 128, 128) and r.data == t.data_ptr() + 8 * 128 * 4
    r = ice.rows(torch.zeros(2, 3, 7, 128).transpose(1, 2))
    assert (r.batch, r.token, r.head) == (3 * 7 * 128, 128, 7 * 128)
