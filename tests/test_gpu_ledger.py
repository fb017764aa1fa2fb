"""The page ledger on the GPU against the same operations on plain lists, one
row after another: forks, growing with copy on write, shrinking, freeing, and
what the kernels refuse."""
import random

import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import serve_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class State:
    def __init__(self, rows, entries, page, n_pages, layers=2, kv_heads=1, head_dim=64):
        self.desc = kvc.make_paged_desc(layers, kv_heads, kv_heads, head_dim, page, n_pages)
        self.pool = torch.zeros(self.desc.pool_shape, dtype=torch.int16, device=DEV)
        self.pool.random_(-30000, 30000)
        self.want = self.pool.clone()
        self.page = page
        self.plain = serve_ref.Ledger([[-7] * entries for _ in range(rows)], [0] * rows,
                                      [0] * n_pages, page)
        self.ledger = kvc.PageLedger(self.desc, _i32(self.plain.table), _i32(self.plain.lens))

    def fork(self, src, dst):
        self.plain.fork(src, dst)
        kvc.fork_async(self.ledger, _i32(src), _i32(dst))

    def resize(self, lens):
        self.plain.copies = []
        self.plain.resize(lens)
        for a, b, n in self.plain.copies:
            p = self.page
            self.want[:, :, b * p:b * p + n] = self.want[:, :, a * p:a * p + n]
        kvc.resize_async(self.ledger, self.pool, _i32(lens))

    def check(self):
        kvc.read_status(self.ledger.status, "ledger")
        assert self.ledger.lens.tolist() == self.plain.lens
        assert self.ledger.refs.tolist() == self.plain.refs
        assert self.ledger.table.tolist() == self.plain.table
        assert torch.equal(self.pool, self.want)


@pytest.mark.parametrize("rows,entries,page,n_pages", [
    (6, 8, 16, 40), (40, 30, 5, 900), (3, 50, 1, 160), (7, 3, 100, 25), (70, 6, 16, 20000),
    (1300, 4, 3, 6000)])
def test_random_histories(rows, entries, page, n_pages):
    rng = random.Random(rows)
    st = State(rows, entries, page, n_pages)
    top = entries * page
    for step in range(12):
        lens = list(st.plain.lens)
        for r in range(rows):
            c = rng.random()
            if c < 0.3:
                lens[r] = rng.randrange(0, top + 1)
            elif c < 0.6:
                lens[r] = min(top, lens[r] + rng.randrange(1, 4))
            elif c < 0.7:
                lens[r] = 0
        # what fits: every row counted with pages of its own
        while sum((n + page - 1) // page for n in lens) > n_pages:
            lens[rng.randrange(rows)] = 0
        if sum((n + page - 1) // page + 1 for n in lens) > n_pages:
            continue
        st.resize(lens)
        st.check()
        order = list(range(rows))
        rng.shuffle(order)
        n = rng.randrange(1, rows)
        src_of = order[n:]
        dst = order[:min(n, 1 + rows // 3)]
        src = [rng.choice(src_of + [-1]) for _ in dst]
        st.fork(src, dst)
        st.check()
    st.resize([0] * rows)
    st.check()
    assert not bool(st.ledger.refs.any())


def test_copy_on_write_of_the_sharers():
    """Three rows share a partly filled page: as they grow in one call, the
    first two take copies and the last keeps it; a row outside the call keeps
    its own too."""
    st = State(5, 4, 16, 30)
    st.resize([21, 0, 0, 0, 0])
    st.fork([0, 0, 0], [1, 2, 4])
    st.check()
    assert st.plain.refs[1] == 4
    st.resize([22, 40, 30, 0, 21])
    st.check()
    assert len(st.plain.copies) == 3 and st.plain.refs[1] == 1
    st.fork([4], [0])
    st.resize([22, 40, 30, 0, 22])  # both holders grow: one copy
    st.check()
    assert len(st.plain.copies) == 1
    # shrinking into a shared page and growing again
    st.fork([1], [3])
    st.resize([0, 20, 30, 33, 22])
    st.check()
    st.resize([16, 32, 32, 48, 22])
    st.check()


def test_large_pages_and_many_layers():
    st = State(9, 2, 1500, 30, layers=7, kv_heads=3, head_dim=96)
    st.resize([1499, 700, 1500, 0, 0, 0, 0, 0, 0])
    st.fork([0, 1, 2, 0, 1], [3, 4, 5, 6, 7])
    st.resize([1500, 701, 1501, 3000, 1499, 1502, 1499, 1500, 1])
    st.check()


def test_capacity():
    st = State(4, 10, 16, 12)
    st.resize([100, 30, 0, 0])  # 7 + 2 pages
    st.check()
    before = st.ledger.refs.clone(), st.ledger.table.clone()
    kvc.resize_async(st.ledger, st.pool, _i32([100, 30, 64, 0]))  # 4 of 3
    assert int(st.ledger.status.item()) == kvc.ERR_CAPACITY
    st.ledger.status.zero_()
    assert torch.equal(st.ledger.refs, before[0]) and torch.equal(st.ledger.table, before[1])
    assert st.ledger.lens.tolist() == [100, 30, 0, 0]
    # rows that shrink in the same call are shrunk first, which makes room
    st.resize([80, 30, 64, 0])
    st.check()
    assert st.plain.refs.count(0) == 1
    kvc.resize_async(st.ledger, st.pool, _i32([0, 30, 64, 150]))  # 10 of 6: the shrunk stay so
    assert int(st.ledger.status.item()) == kvc.ERR_CAPACITY
    assert st.ledger.lens.tolist() == [0, 30, 64, 0]


def test_fork_errors():
    for src, dst, done in (([0, 0], [2, 2], ()), ([0, 2], [2, 3], ()), ([0], [0], ()),
                           ([4, 0], [2, 3], (1,)), ([0, 1], [-1, 3], (1,)),
                           ([0, 1], [4, 2], (1,)), ([0, 1, 0], [2, 3, 2], (1,))):
        st = State(4, 4, 16, 20)
        st.resize([40, 17, 5, 0])
        kvc.fork_async(st.ledger, _i32(src), _i32(dst))
        assert int(st.ledger.status.item()) == kvc.ERR_SHAPE
        st.ledger.status.zero_()
        st.plain.fork([src[i] for i in done], [dst[i] for i in done])
        st.check()
    # a length outside the table, a bad page id, a page that nobody holds
    st = State(4, 4, 16, 20)
    st.resize([40, 17, 5, 0])
    for name in ("lens", "id", "free"):
        if name == "lens":
            st.ledger.lens[0] = 65
        elif name == "id":
            st.ledger.lens[0] = 40
            st.ledger.table[0, 1] = 20
        else:
            st.ledger.table[0, 1] = 19
        kvc.fork_async(st.ledger, _i32([1]), _i32([0])) if name != "lens" else \
            kvc.fork_async(st.ledger, _i32([0]), _i32([3]))
        assert int(st.ledger.status.item()) == kvc.ERR_SHAPE
        st.ledger.status.zero_()
        if name == "id":
            assert st.ledger.lens[0] == 17
            st.ledger.lens[0] = 40
            st.ledger.refs[int(st.ledger.table[1, 0])] += 0
    assert bool((st.ledger.refs >= 0).all())


def test_resize_errors():
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        st = State(4, 4, 16, 20)
        st.resize([40, 17, 5, 0])
        kvc.resize_async(st.ledger, st.pool, _i32([40, bad, 20, 3]))
        assert int(st.ledger.status.item()) == kvc.ERR_SHAPE
        st.ledger.status.zero_()
        st.resize([40, 17, 20, 3])  # the others were resized: nothing left to do
        st.check()
    st = State(2, 4, 16, 20)
    st.resize([40, 17])
    st.ledger.table[0, 2] = -1  # the page to grow out of
    kvc.resize_async(st.ledger, st.pool, _i32([41, 17]))
    assert int(st.ledger.status.item()) == kvc.ERR_SHAPE
    st.ledger.status.zero_()
    kvc.resize_async(st.ledger, st.pool, _i32([0, 17]))  # and to release
    assert int(st.ledger.status.item()) == kvc.ERR_SHAPE
    assert bool((st.ledger.refs >= 0).all())


def test_the_ledgers_tensors_are_read_at_each_call():
    st = State(4, 4, 16, 12)
    st.resize([20, 5, 0, 33])
    st.check()
    old = [getattr(st.ledger, k) for k in ("table", "lens", "refs")]
    before = [t.clone() for t in old]
    for k, t in zip(("table", "lens", "refs"), old):
        setattr(st.ledger, k, t.clone())
    st.fork([0], [2])
    st.resize([21, 40, 22, 0])
    st.check()
    assert all(torch.equal(a, b) for a, b in zip(old, before))


def test_forked_sequences_decode_apart():
    """A restored context forked three ways: each continuation appends its own
    token and attends; all read the shared pages and none another's token."""
    heads, kv_heads, dim, page, m = 8, 2, 64, 16, 53
    desc = kvc.make_paged_desc(1, heads, kv_heads, dim, page, 20)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    flat = torch.randn((1, 2, m, kv_heads * dim), generator=g, device=DEV).half()
    pool = torch.full(desc.pool_shape, float("nan"), dtype=torch.float16, device=DEV)
    table, lens = torch.full((4, 6), -1, dtype=torch.int32, device=DEV), _i32([0, 0, 0, 0])
    ledger = kvc.PageLedger(desc, table, lens)
    kvc.resize_async(ledger, pool, _i32([m, 0, 0, 0]))
    kvc.page_in_async(desc, flat, 0, pool, table[0], 0, m, ledger.status)
    kvc.fork_async(ledger, _i32([0, 0, 0]), _i32([1, 2, 3]))
    kvc.resize_async(ledger, pool, _i32([m + 1] * 4))
    batch = kvc.PagedBatch(table, lens)
    wsp = kvc.PagedWorkspace(desc, batch)
    q = torch.randn((4, heads, dim), generator=g, device=DEV).half()
    k, v = (torch.randn((4, kv_heads, dim), generator=g, device=DEV).half() for _ in range(2))
    kvc.append_async(desc, batch, 0, pool, k, v, wsp)
    out = torch.empty_like(q)
    kvc.attend_async(desc, batch, 0, pool, q, out, wsp)
    kvc.read_status(wsp.status, "step")
    kvc.read_status(ledger.status, "ledger")
    assert sorted(ledger.refs.tolist())[-4:] == [1, 4, 4, 4]
    for r in range(4):
        kk = torch.cat([flat[0, 0].view(m, kv_heads, dim), k[r:r + 1]])
        vv = torch.cat([flat[0, 1].view(m, kv_heads, dim), v[r:r + 1]])
        import paged_ref as ref

        o, _, bound, _ = ref.attend(q[r:r + 1], kk, vv, [m], dim ** -0.5, 0, torch.float16,
                                    torch.float16)
        assert bool(((out[r:r + 1].double() - o).abs() <= bound).all())


def test_captured_and_replayed():
    st = State(12, 6, 16, 300)
    st.resize([30 + r if r < 4 else 0 for r in range(12)])
    src, dst, lens = _i32([0, 1, 2, 3, 0, -1]), _i32([4, 5, 6, 7, 8, 9]), _i32([0] * 12)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        kvc.fork_async(st.ledger, src, dst)
        kvc.resize_async(st.ledger, st.pool, lens)
    for step in range(4):
        src_host = [(i + step) % 4 for i in range(5)] + [-1]
        src.copy_(_i32(src_host))
        plain = st.plain
        plain.fork(src_host, [4, 5, 6, 7, 8, 9])
        target = [n + (1 + step if n else 0) for n in plain.lens]
        plain.copies = []
        plain.resize(target)
        for a, b, n in plain.copies:
            st.want[:, :, b * 16:b * 16 + n] = st.want[:, :, a * 16:a * 16 + n]
        lens.copy_(_i32(target))
        graph.replay()
        torch.cuda.synchronize()
        st.check()


def test_pages_past_four_giga_elements():
    """Copy on write, a tree's attention and its kept path in pages whose
    elements pass 2^32, against the same in a small pool."""
    heads, kv_heads, dim, page, m, n = 16, 8, 128, 16, 75, 12
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    flat = torch.randn((1, 2, m + n, kv_heads * dim), generator=g, device=DEV).half()
    q = torch.randn((2 * n, heads, dim), generator=g, device=DEV).half()
    parent = _i32([max(i - 1 - i % 3, -1) for i in range(n)] * 2)
    results = []
    for n_pages in (20, 280000):
        desc = kvc.make_paged_desc(1, heads, kv_heads, dim, page, n_pages)
        pool = torch.empty(desc.pool_shape, dtype=torch.float16, device=DEV)
        refs = torch.ones(n_pages, dtype=torch.int32, device=DEV)
        refs[-20:] = 0
        table, lens = torch.full((2, 8), -1, dtype=torch.int32, device=DEV), _i32([0, 0])
        ledger = kvc.PageLedger(desc, table, lens, refs)
        kvc.resize_async(ledger, pool, _i32([m, 0]))
        kvc.page_in_async(desc, flat, 0, pool, table[0], 0, m, ledger.status)
        kvc.fork_async(ledger, _i32([0]), _i32([1]))
        kvc.resize_async(ledger, pool, _i32([m + n] * 2))
        batch = kvc.PagedBatch(table, lens, q_start=_i32([0, n, 2 * n]))
        tree = kvc.Tree(parent, n)
        wsp = kvc.PagedWorkspace(desc, batch, 2 * n, tree=tree)
        kvc.tree_async(desc, batch, tree, wsp)
        kv = flat[0, :, m:].view(2, n, kv_heads, dim).repeat(1, 2, 1, 1)
        kvc.append_async(desc, batch, 0, pool, kv[0], kv[1], wsp, tree=tree)
        out = torch.empty_like(q)
        kvc.attend_tree_async(desc, batch, tree, 0, pool, q, out, wsp)
        new_lens = _i32([0, 0])
        kvc.keep_async(desc, batch, pool, _i32([[0, 5, 11], [2, 3, 4]]), _i32([3, 3]), new_lens,
                       2 * n, wsp.status)
        kvc.read_status(wsp.status, "far")
        kvc.read_status(ledger.status, "far")
        rows = []
        for b in range(2):
            got = torch.empty((1, 2, m + 3, kv_heads * dim), dtype=torch.float16, device=DEV)
            kvc.page_out_async(desc, pool, table[b], 0, m + 3, got, 0, ledger.status)
            rows.append(got)
            want = torch.cat([flat[:, :, :m], flat[:, :, [m + t for t in
                                                          ([0, 5, 11], [2, 3, 4])[b]]]], 2)
            assert torch.equal(got, want)
        assert int(table[0, 0]) == n_pages - 20 and len(set(table[:, 4].tolist())) == 2
        results.append((out, *rows))
        del pool
    for a, b in zip(*results):
        assert torch.equal(a, b)
