"""CPU checks of the calls around normed heads, sinks, drafted trees and shared
pages: struct layouts and every refusal that the header documents (returned
before anything is launched), and the binding's own checks."""
import ctypes
import os

import pytest
import torch

import kv_cache_compression_decode_amd as kvc
from test_paged_host import A, BATCH_BAD, _batch, _desc

INVALID, SHAPE, CAPACITY = kvc.ERR_INVALID_ARG, kvc.ERR_SHAPE, kvc.ERR_CAPACITY


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kvc.LIB_PATH):
        from kv_cache_compression_decode_amd import build

        build.build()
    return kvc.lib()


def test_struct_layouts():
    assert ctypes.sizeof(kvc._HeadNormArgs) == 24
    assert ctypes.sizeof(kvc._TreeArgs) == 32
    assert ctypes.sizeof(kvc._LedgerArgs) == 32


def _trees(**kw):
    return _batch(**{"q_start": A, "n_tokens": 9, **kw})


def _tree(parent=A, mask=A, depth=A, most=8, reserved=0):
    return kvc._TreeArgs(parent, mask, depth, most, reserved)


def _norm(q=A, k=A, eps=1e-6, reserved=0):
    return kvc._HeadNormArgs(q, k, eps, reserved)


def _append(L, d=None, b=None, layer=0, pool=A, k=A, ks=256, v=A, vs=256, q=A, qs=1024, o=A,
            os_=1024, rope=None, norm=None, depth=None, status=A):
    return L.kvc_append_norm(d or _desc(), b or _batch(), layer, pool, k, ks, v, vs, q, qs, o, os_,
                             rope, norm, depth, status, None)


def _sinks(L, d=None, b=None, layer=0, pool=A, q=A, qs=1024, scale=1.0, window=5, sinks=2, o=A,
           os_=1024, lse=A, ws=A, ws_bytes=1 << 40, status=A):
    return L.kvc_attend_sinks(d or _desc(), b or _batch(), layer, pool, q, qs, scale, window, sinks,
                              o, os_, lse, ws, ws_bytes, status, None)


def _attend_tree(L, d=None, b=None, tree=None, layer=0, pool=A, q=A, qs=1024, scale=1.0, o=A,
                 os_=1024, lse=A, ws=A, ws_bytes=1 << 40, status=A):
    return L.kvc_attend_tree(d or _desc(), b or _trees(), tree or _tree(), layer, pool, q, qs,
                             scale, o, os_, lse, ws, ws_bytes, status, None)


def _build(L, d=None, b=None, tree=None, status=A):
    return L.kvc_tree_build(d or _desc(), b or _trees(), tree or _tree(), status, None)


def _keep(L, d=None, b=None, pool=A, path=A, stride=4, kept=A, new_lens=2 * A, status=A):
    return L.kvc_keep(d or _desc(), b or _trees(), pool, path, stride, kept, new_lens, status, None)


def _ledger(table=A, lens=A, refs=A, rows=5, stride=10):
    return kvc._LedgerArgs(table, lens, refs, rows, stride)


def _fork(L, d=None, g=None, src=A, dst=A, n=3, status=A):
    return L.kvc_fork(d or _desc(), g or _ledger(), src, dst, n, status, None)


def _resize(L, d=None, g=None, lens=A, pool=A, ws=A, ws_bytes=1 << 30, status=A):
    return L.kvc_resize(d or _desc(), g or _ledger(), lens, pool, ws, ws_bytes, status, None)


@pytest.mark.parametrize("bad", [
    dict(n_layers=0), dict(n_heads=9), dict(head_dim=80), dict(page_tokens=0), dict(n_pages=0),
    dict(page_tokens=1 << 16, n_pages=1 << 15), dict(cache_dtype=1, io_dtype=0)])
def test_descriptor_refusals(L, bad):
    d = _desc(**bad)
    for call in (_append, _sinks, _attend_tree, _build, _keep, _fork, _resize):
        assert call(L, d) == INVALID, call
    assert L.kvc_attend_tree_ws_bytes(d, _trees(), _tree()) == 0
    assert L.kvc_resize_ws_bytes(d) == 0


@pytest.mark.parametrize("bad,code", BATCH_BAD)
def test_batch_refusals(L, bad, code):
    b = _batch(**bad)
    assert _append(L, b=b) == code and _sinks(L, b=b) == code
    if b.q_start:
        assert _attend_tree(L, b=b) == code and _keep(L, b=b) == code


def test_append_norm_refusals(L):
    assert _append(L, layer=2, norm=_norm()) == SHAPE
    for p in ("pool", "k", "v", "status"):
        assert _append(L, **{p: None}) == INVALID and _append(L, **{p: A + 2}) == INVALID
    for p in ("q", "o"):
        assert _append(L, **{p: None}) == INVALID and _append(L, **{p: A + 8}) == INVALID
    assert _append(L, qs=2048) == SHAPE
    for n in (_norm(k=None), _norm(q=None), _norm(k=A + 8), _norm(q=A + 4), _norm(reserved=1),
              _norm(eps=0.0), _norm(eps=-1e-6), _norm(eps=float("inf")), _norm(eps=float("nan")),
              _norm(eps=1e-40)):
        assert _append(L, norm=n) == INVALID
    assert _append(L, depth=A + 2) == INVALID
    bad_rope = kvc._RopeArgs(A, 200, 24, 0, 0)
    assert _append(L, norm=_norm(), rope=bad_rope) == INVALID


def test_sinks_refusals(L):
    assert _sinks(L, layer=2) == SHAPE
    for p in ("pool", "q", "o", "status"):
        assert _sinks(L, **{p: None}) == INVALID and _sinks(L, **{p: A + 2}) == INVALID
    assert _sinks(L, lse=A + 2) == INVALID and _sinks(L, scale=float("nan")) == INVALID
    long = _batch(table_stride=10000, max_len=100000)
    need = L.kvc_attend_ws_bytes(_desc(), long)
    assert _sinks(L, b=long, ws_bytes=need - 1) == CAPACITY
    assert _sinks(L, b=long, ws=None) == INVALID
    assert L.kvc_attend_sinks(_desc(), None, 0, A, A, 1024, 1.0, 5, 2, A, 1024, A, A, 1 << 40, A,
                              None) == INVALID


def test_tree_refusals(L):
    assert _build(L, b=_batch()) == INVALID and _attend_tree(L, b=_batch()) == INVALID
    for t in (_tree(most=0), _tree(most=4097), _tree(reserved=1)):
        assert _build(L, tree=t) == INVALID and _attend_tree(L, tree=t) == INVALID
        assert L.kvc_attend_tree_ws_bytes(_desc(), _trees(), t) == 0
    for t in (_tree(parent=None), _tree(mask=None), _tree(depth=None), _tree(parent=A + 2),
              _tree(mask=A + 4), _tree(depth=A + 1)):
        assert _build(L, tree=t) == INVALID
    for t in (_tree(mask=None), _tree(mask=A + 4)):
        assert _attend_tree(L, tree=t) == INVALID
    assert _build(L, status=None) == INVALID and _build(L, status=A + 2) == INVALID
    assert _build(L, b=_trees(q_start=A + 2)) == INVALID
    for p in ("pool", "q", "o", "status"):
        assert _attend_tree(L, **{p: None}) == INVALID
        assert _attend_tree(L, **{p: A + 2}) == INVALID
    assert _attend_tree(L, layer=2) == SHAPE
    long = _trees(table_stride=10000, max_len=100000)
    need = L.kvc_attend_tree_ws_bytes(_desc(), long, _tree())
    assert need > 0
    assert _attend_tree(L, b=long, ws_bytes=need - 1) == CAPACITY
    assert _attend_tree(L, b=long, ws=None) == INVALID
    assert _attend_tree(L, b=long, ws=A + 128) == INVALID
    big = _trees(n_tokens=1 << 20)
    assert _attend_tree(L, d=_desc(n_heads=16), b=big, qs=2048, os_=2048) == SHAPE


def test_keep_refusals(L):
    assert _keep(L, b=_batch()) == INVALID
    assert _keep(L, stride=4097) == SHAPE
    for p in ("pool", "path", "kept", "new_lens", "status"):
        assert _keep(L, **{p: None}) == INVALID and _keep(L, **{p: A + 2}) == INVALID
    for at in (A, A + 4, A + 8, A - 8):  # lens, kept and path: three entries at A
        assert _keep(L, new_lens=at, kept=4 * A, path=5 * A) == SHAPE
        assert _keep(L, b=_trees(lens=3 * A), new_lens=at, path=5 * A) == SHAPE
        assert _keep(L, b=_trees(lens=3 * A), new_lens=at, kept=4 * A) == SHAPE
    # q_start: 4 entries at 6 A; the table: 3 * 10 at 7 A
    apart = dict(lens=3 * A, q_start=6 * A, table=7 * A, table_stride=10)
    for at in (6 * A - 8, 6 * A + 12, 7 * A - 8, 7 * A + 116):
        assert _keep(L, b=_trees(**apart), new_lens=at, kept=4 * A, path=5 * A) == SHAPE
    # the last of path's 3 * 4 entries
    assert _keep(L, b=_trees(lens=3 * A), new_lens=A + 44, kept=4 * A) == SHAPE
    wide = _desc(n_layers=32767, n_heads=4096, n_kv_heads=4096, head_dim=256, page_tokens=1)
    assert _keep(L, d=wide) == SHAPE


def test_ledger_refusals(L):
    for call in (_fork, _resize):
        assert call(L, g=_ledger(rows=2049)) == SHAPE
        for p in ("table", "lens", "refs"):
            assert call(L, g=_ledger(**{p: None})) == INVALID
            assert call(L, g=_ledger(**{p: A + 2})) == INVALID
        assert call(L, status=None) == INVALID and call(L, status=A + 2) == INVALID
    assert _fork(L, n=2049) == SHAPE
    for p in ("src", "dst"):
        assert _fork(L, **{p: None}) == INVALID and _fork(L, **{p: A + 2}) == INVALID
    for p in ("lens", "pool", "ws"):
        assert _resize(L, **{p: None}) == INVALID and _resize(L, **{p: A + 2}) == INVALID
    need = L.kvc_resize_ws_bytes(_desc())
    assert need > 0 and _resize(L, ws_bytes=need - 1) == CAPACITY
    assert L.kvc_fork(_desc(), None, A, A, 3, A, None) == INVALID
    assert L.kvc_resize(_desc(), None, A, A, A, 1 << 30, A, None) == INVALID


def test_empty_calls_do_nothing(L):
    none = _batch(n_seqs=0, n_tokens=0, table=None, lens=None)
    trees = _batch(n_seqs=0, n_tokens=0, table=None, lens=None, q_start=A)
    assert _append(L, b=none, norm=_norm()) == 0 and _sinks(L, b=none) == 0
    assert _build(L, b=trees) == 0 and _attend_tree(L, b=trees) == 0
    assert _keep(L, b=trees, path=None, stride=0, kept=None) == 0
    assert _fork(L, n=0, src=None, dst=None) == 0
    nothing = _ledger(None, None, None, 0, 0)
    assert _fork(L, g=nothing, n=0) == 0 and _resize(L, g=nothing, lens=None, ws=None) == 0


@pytest.mark.parametrize("head_dim", [64, 96, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (64, 8), (128, 1), (6, 2), (4096, 4096)])
def test_tree_workspace_bound(L, head_dim, heads, kv_heads):
    """The documented bound holds for every batch."""
    d = _desc(n_heads=heads, n_kv_heads=kv_heads, head_dim=head_dim)
    for seqs in (1, 3, 17, 64, 700):
        for most in (1, 2, 4, 16, 33, 100, 1000):
            for tokens in (seqs, seqs * ((most + 1) // 2), seqs * most):
                for length in (100, 3000, 100000, 1 << 30):
                    b = _trees(n_seqs=seqs, n_tokens=tokens, table_stride=1 << 27, max_len=length)
                    n = L.kvc_attend_tree_ws_bytes(d, b, _tree(most=most))
                    assert n <= 131072 * (4 * head_dim + 8) + 131584


def test_binding_refusals():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        kvc.Tree(i, 4)
    with pytest.raises(ValueError):
        kvc.HeadNorm(torch.ones(64), torch.ones(64))
    d = kvc.make_paged_desc(1, 8, 2, 64, 16, 4)
    with pytest.raises(ValueError):
        kvc.PageLedger(d, torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
