"""CPU checks of the binding where a program replaces the fields of what it
keeps (a ledger's, a tree's, a norm's tensors): what does not fit is refused
before anything is launched."""
import os

import pytest
import torch

import kv_cache_compression_decode_amd as kvc

CPU = torch.device("cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(kvc.LIB_PATH):
        from kv_cache_compression_decode_amd import build

        build.build()


class Stand(torch.Tensor):
    """A host tensor that says it is on the GPU: refused calls never touch it."""
    is_cuda = True


def _t(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Stand)


def _elsewhere(t):
    return torch.zeros(t.shape, dtype=t.dtype, device="meta").as_subclass(Stand)


def _bad_int32(t):
    """The same entries in another type, with gaps, with a dimension more, on
    another device."""
    wide = _t(*t.shape[:-1], 2 * t.shape[-1])[..., ::2]
    return [t.long().as_subclass(Stand), wide, t[None], _elsewhere(t)]


@pytest.fixture
def ledger():
    return kvc.PageLedger(kvc.make_paged_desc(1, 2, 2, 64, 16, 40), _t(5, 8), _t(5), _t(40))


def _ledger_refuses(g, new_lens=None):
    pool = torch.zeros(g.desc.pool_shape, dtype=torch.float16)
    with pytest.raises(ValueError):
        kvc.fork_async(g, _t(2), _t(2))
    with pytest.raises(ValueError):
        kvc.resize_async(g, pool, _t(g.lens.shape[0]) if new_lens is None else new_lens)


def test_ledger_sizes(ledger):
    for field, t in (("table", _t(6, 8)), ("table", _t(4, 8)), ("lens", _t(6)), ("lens", _t(4)),
                     ("refs", _t(39)), ("refs", _t(41)), ("refs", _t(0))):
        kept = getattr(ledger, field)
        setattr(ledger, field, t)
        _ledger_refuses(ledger)
        setattr(ledger, field, kept)
    ledger.desc = kvc.make_paged_desc(1, 2, 2, 64, 16, 41)  # refs has 40 entries
    _ledger_refuses(ledger)


def test_ledger_types(ledger):
    for field in ("table", "lens", "refs"):
        kept = getattr(ledger, field)
        for t in _bad_int32(kept):
            setattr(ledger, field, t)
            _ledger_refuses(ledger, _t(5))
        setattr(ledger, field, kept)


def test_ledger_grows(ledger):
    """Replaced one after another by larger ones that fit: accepted."""
    ledger.table = _t(9, 30)
    ledger.lens = _t(9)
    a = ledger._args()
    assert (a.n_rows, a.table_stride) == (9, 30)
    with pytest.raises(ValueError):  # new lengths of the rows before
        kvc.resize_async(ledger, torch.zeros(ledger.desc.pool_shape, dtype=torch.float16), _t(5))


def _tree():
    return kvc.Tree(_t(9), 70)


def _fields(tree):
    tree.mask, tree.depth = tree.mask.as_subclass(Stand), tree.depth.as_subclass(Stand)
    return tree


def test_tree():
    _fields(_tree())._check(9, CPU)
    for field, t in (("max_tokens", 129), ("max_tokens", 64), ("max_tokens", 0),
                     ("max_tokens", 5000), ("mask", _t(9, 1, dtype=torch.int64)),
                     ("mask", _t(8, 2, dtype=torch.int64)), ("mask", _t(18, dtype=torch.int64)),
                     ("mask", _t(9, 2)), ("mask", _t(9, 4, dtype=torch.int64)[:, ::2]),
                     ("mask", torch.zeros((9, 2), dtype=torch.int64)),
                     ("mask", _elsewhere(_t(9, 2, dtype=torch.int64))),
                     ("depth", _t(8)), ("depth", _t(10)), ("parent", _t(8)), ("parent", _t(10)),
                     *(("depth", t) for t in _bad_int32(_t(9))),
                     *(("parent", t) for t in _bad_int32(_t(9)))):
        tree = _fields(_tree())
        setattr(tree, field, t)
        with pytest.raises(ValueError):
            tree._check(9, CPU)


def test_tree_calls_check():
    """The calls with a tree come to its check before anything else of it."""
    desc = kvc.make_paged_desc(1, 2, 2, 64, 16, 40)
    batch = kvc.PagedBatch(_t(2, 8), _t(2), q_start=_t(3))
    pool = torch.zeros(desc.pool_shape, dtype=torch.float16)
    tree = _fields(_tree())
    wsp = kvc.PagedWorkspace(desc, batch, 9, tree=tree)
    q = torch.zeros((9, 2, 64), dtype=torch.float16)
    tree.max_tokens = 129
    for call in (lambda: kvc.tree_async(desc, batch, tree, wsp),
                 lambda: kvc.append_async(desc, batch, 0, pool, q, q, wsp, tree=tree),
                 lambda: kvc.attend_tree_async(desc, batch, tree, 0, pool, q, q, wsp)):
        with pytest.raises(ValueError, match="mask must be"):
            call()


def test_head_norm():
    desc = kvc.make_paged_desc(1, 2, 2, 64, 16, 40)
    batch = kvc.PagedBatch(_t(9, 8), _t(9))
    pool = torch.zeros(desc.pool_shape, dtype=torch.float16)
    wsp = kvc.PagedWorkspace(desc, batch)
    q = torch.zeros((9, 2, 64), dtype=torch.float16)

    def f32(n):
        return _t(n, dtype=torch.float32)

    for field in ("q_weight", "k_weight"):
        for t in (f32(63), f32(65), f32(128)[::2], _t(64, dtype=torch.float16), f32(64)[None],
                  _elsewhere(f32(64))):
            norm = kvc.HeadNorm(f32(64), f32(64))
            setattr(norm, field, t)
            with pytest.raises(ValueError, match="norms' weights"):
                kvc.append_async(desc, batch, 0, pool, q, q, wsp, norm=norm)
