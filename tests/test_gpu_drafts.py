"""Drafted trees on the GPU against plain forms: the tree's mask and depths,
appending with norms at the depths' positions, attention of the tree's tokens,
and keeping an accepted path; and all of them together as a decoding step."""
import random

import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import paged_ref as ref
import serve_ref
from test_gpu_paged import BF16, DEV, F16, Setup

pytestmark = pytest.mark.gpu


def _tree(n, kind, seed=0):
    rng = random.Random(seed * 1000 + n)
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    return [rng.randrange(max(-1, i - 12), i) for i in range(n)]


class Drafts(Setup):
    def __init__(self, lens, new, *shape, kind="random", max_tokens=None, seed=1, **kw):
        super().__init__(lens, new, *shape, seed=seed, **kw)
        self.parents = [_tree(n, kind, seed + b) for b, n in enumerate(new)]
        flat = [p for t in self.parents for p in t] + [5] * (self.n_tok - self.start[-1])
        self.tree = kvc.Tree(torch.tensor(flat, dtype=torch.int32, device=DEV),
                             max_tokens or max(new + [1]))
        self.wsp = kvc.PagedWorkspace(self.desc, self.batch, self.n_tok, tree=self.tree)
        kvc.tree_async(self.desc, self.batch, self.tree, self.wsp)
        kvc.read_status(self.wsp.status, "tree")

    def seen(self, b):
        m, n = self.lens_host[b], self.new_host[b]
        seen = torch.zeros((n, m), dtype=torch.bool)
        see = torch.tensor(serve_ref.ancestors(self.parents[b]), dtype=torch.bool).view(n, n)
        for i in range(n):
            if m - n + i < 0:
                continue  # padding
            for t in range(n):
                if m - n + t >= 0:
                    seen[i, m - n + t] = see[i, t]
            seen[i, : max(m - n, 0)] = True
        return seen.to(DEV)

    def attend(self):
        out = torch.full((self.n_tok, self.heads, self.head_dim), 7.0, dtype=self.io, device=DEV)
        lse = torch.full((self.n_tok, self.heads), 7.0, device=DEV)
        kvc.attend_tree_async(self.desc, self.batch, self.tree, 1, self.pool, self.q, out,
                              self.wsp, lse=lse)
        kvc.read_status(self.wsp.status, "attend_tree")
        return out, lse

    def check(self, out, lse, skip=()):
        for b, n in enumerate(self.new_host):
            if n == 0:
                continue
            a = self.start[b]
            k, v = self.cached(b)
            seen = self.seen(b)
            # 11: the bound of the larger tiles, which holds for the smaller ones too
            o, e, bo, be = serve_ref.attend_seen(self.q[a:a + n], k, v, seen, self.head_dim ** -0.5,
                                                 self.cache, self.io, 11)
            for i in range(n):
                if (b, i) in skip:
                    continue
                got, got_e = out[a + i].double(), lse[a + i].double()
                if not bool(seen[i].any()):
                    assert bool((got == 0).all()) and bool((got_e == float("-inf")).all())
                    continue
                assert bool(((got - o[i]).abs() <= bo[i]).all()), (b, i)
                assert bool(((got_e - e[i]).abs() <= be[i]).all()), (b, i)
        a = self.start[-1]
        assert bool((out[a:] == 7.0).all()) and bool((lse[a:] == 7.0).all())


# -------------------------------------------------------------------- tree
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("most", [None, 200, 4096])
def test_tree_mask_and_depth(kind, most):
    new = [1, 63, 0, 64, 65, 130, 7]
    st = Drafts([n + 5 for n in new], new, 4, 2, 64, 16, F16, F16, kind=kind, max_tokens=most,
                spare=3)
    words = st.tree.mask.shape[1]
    mask = st.tree.mask.cpu().tolist()
    depth = st.tree.depth.cpu().tolist()
    for b, p in enumerate(st.parents):
        see = serve_ref.ancestors(p)
        assert depth[st.start[b]:st.start[b + 1]] == serve_ref.depths(p)
        for i, row in enumerate(see):
            bits = sum(1 << t for t, s in enumerate(row) if s)
            got = sum((w & (2 ** 64 - 1)) << (64 * k)
                      for k, w in enumerate(mask[st.start[b] + i]))
            assert got == bits
    assert mask[st.start[-1]:] == [[0] * words] * 3 and depth[st.start[-1]:] == [0] * 3


def test_tree_errors():
    st = Drafts([20, 20], [4, 6], 4, 2, 64, 16, F16, F16, kind="chain")
    for at, value in ((5, 1), (5, 7), (4, -2), (0, 2 ** 31 - 1), (9, -2 ** 31)):
        parent = st.tree.parent.clone()
        parent[at] = value
        tree = kvc.Tree(parent, 6)
        kvc.tree_async(st.desc, st.batch, tree, st.wsp)
        assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
        st.wsp.status.zero_()
        # it counts as a root: what does not follow it is as before
        good = [i for i in range(10) if not (at <= i < (4 if at < 4 else 10))]
        assert torch.equal(tree.depth[good], st.tree.depth[good])
        assert int(tree.depth[at]) == 0
    tree = kvc.Tree(st.tree.parent, 5)  # the second sequence has 6
    kvc.tree_async(st.desc, st.batch, tree, st.wsp)
    assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
    assert torch.equal(tree.depth[:4], st.tree.depth[:4]) and not bool(tree.mask[4:].any())


# ------------------------------------------------------------ attention
TREES = [
    # heads, kv_heads, head_dim, page, io, cache, lens, new
    (8, 2, 64, 16, F16, F16, [40, 100, 33], [5, 3, 33]),
    (4, 4, 128, 16, BF16, BF16, [130, 1, 200, 513], [8, 1, 2, 5]),
    (64, 8, 128, 16, F16, F16, [1526], [26]),
    (64, 8, 128, 20, BF16, F16, [900, 0, 65, 64], [60, 2, 65, 64]),
    (6, 2, 256, 7, F16, F16, [400, 90, 300], [50, 33, 4]),
    (5, 5, 96, 16, F16, F16, [600, 300], [150, 7]),
    (8, 1, 64, 10, BF16, BF16, [300, 150], [150, 150]),
    (40, 1, 128, 1, BF16, F16, [300, 65], [3, 9]),
    (128, 1, 64, 16, F16, F16, [700, 100], [11, 4]),
    # few rows: one and two to a KV head, sixteen, seventeen, thirty-two, thirty-three
    (2, 2, 128, 16, F16, F16, [1300, 64, 7], [1, 2, 1]),
    (8, 8, 128, 32, BF16, BF16, [2100, 900, 0, 16], [16, 9, 3, 16]),
    (4, 4, 64, 16, F16, F16, [1100, 17], [17, 17]),
    (16, 4, 128, 16, BF16, F16, [3000, 31, 700], [8, 7, 4]),
    (3, 3, 96, 5, BF16, BF16, [800, 32], [32, 3]),
    (3, 3, 256, 16, F16, F16, [640, 33], [33, 12]),
    (12, 6, 256, 16, BF16, F16, [1030, 14], [8, 7]),
    (4, 2, 256, 16, F16, F16, [500, 40, 1200], [16, 9, 13]),
    (10, 5, 128, 16, BF16, BF16, [2500, 40, 1200, 16], [16, 9, 13, 16]),
    (24, 1, 128, 16, F16, F16, [5000], [1]),
    # sequences that begin with the tree's tokens, padding among them
    (4, 2, 64, 16, F16, F16, [20, 9, 3], [20, 12, 5]),
    # many sequences
    (4, 2, 64, 16, F16, F16, [(i * 37) % 23 * 20 + 6 for i in range(150)],
     [i % 7 for i in range(150)]),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,new", TREES)
def test_attend_tree(heads, kv_heads, head_dim, page, io, cache, lens, new):
    st = Drafts(lens, new, heads, kv_heads, head_dim, page, io, cache, spare=2)
    st.check(*st.attend())


@pytest.mark.parametrize("head_dim", [64, 96, 128, 256])
@pytest.mark.parametrize("most,group", [(4, 4), (8, 4), (12, 4), (50, 4)])
def test_attend_tree_many_sequences_to_a_piece(head_dim, most, group):
    """Sequences of every length from none to a few tiles, several in each
    workgroup's or wave's share, with long ones between them that are cut."""
    lens = [0, 5, 40, 90, 33, 64, 65, 1, 700, 31, 32, 100, 12, 1500, 95, 47, 16, 63, 130, 2]
    new = [min(m, 1 + (7 * i) % most) if m else i % 3 for i, m in enumerate(lens)]
    new[13] = most
    st = Drafts(lens, new, 2 * group, 2, head_dim, 16, F16, F16)
    st.check(*st.attend())


@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("n,group", [(7, 1), (70, 1), (40, 8)])
def test_attend_tree_shapes(kind, n, group):
    st = Drafts([n + 200, n], [n, n], 2 * group, 2, 64, 16, F16, F16, kind=kind)
    out, lse = st.attend()
    st.check(out, lse)
    if kind == "chain":  # a prompt's rows are the same
        wsp = kvc.PagedWorkspace(st.desc, st.batch, st.n_tok)
        kvc.attend_prompt_async(st.desc, st.batch, 1, st.pool, st.q, out, wsp, lse=lse)
        kvc.read_status(wsp.status, "prompt")
        st.check(out, lse)


@pytest.mark.parametrize("n,group", [(12, 1), (12, 2), (30, 8)])
def test_attend_tree_infinite_sibling(n, group):
    """What stands in a token that a row does not follow has no effect on it."""
    st = Drafts([n + 77], [n], 2 * group, 2, 128, 16, F16, F16, kind="random")
    s = st.slots(0)
    bad = n // 2
    st.pool[1, 1, s[77 + bad]] = float("inf")
    st.pool[1, 1, s[77 + bad], ::3] = float("nan")
    out, lse = st.attend()
    hit = {(0, i) for i in range(n) if serve_ref.ancestors(st.parents[0])[i][bad]}
    assert 0 < len(hit) < n
    st.check(out, lse, skip=hit)
    for _, i in hit:
        assert not bool(torch.isfinite(out[i].double()).any())


def test_attend_tree_errors():
    for damage in ("page", "length", "more", "rows"):
        st = Drafts([300, 100], [6, 9], 4, 2, 64, 16, F16, F16)
        if damage == "page":
            st.table[1, 3] = -1
        elif damage == "length":
            st.lens[0] = 301
        elif damage == "more":
            st.tree.max_tokens = 8
            st.tree.mask = st.tree.mask[:, :1].contiguous()
        else:
            st.batch.q_start[1] = 16
        out = torch.zeros((st.n_tok, 4, 64), dtype=F16, device=DEV)
        kvc.attend_tree_async(st.desc, st.batch, st.tree, 1, st.pool, st.q, out, st.wsp)
        with pytest.raises(kvc.KvcError) as e:
            kvc.read_status(st.wsp.status, "attend_tree")
        assert e.value.code == kvc.ERR_SHAPE


# ---------------------------------------------------------------- append
APPEND = [
    # heads, kv_heads, head_dim, page, io, cache, rotary, interleaved, normed, drafts
    (8, 2, 64, 16, F16, F16, 64, False, True, False),
    (4, 4, 128, 16, BF16, BF16, 128, True, True, True),
    (64, 8, 128, 20, BF16, F16, 64, False, True, True),
    (6, 2, 96, 7, F16, F16, 48, False, True, False),
    (6, 2, 96, 7, BF16, BF16, 96, True, True, True),
    (6, 3, 96, 7, BF16, F16, 32, False, False, True),
    (5, 5, 256, 1, F16, F16, 256, False, True, True),
    (40, 1, 256, 33, BF16, F16, 32, True, True, False),
    (3, 1, 64, 16, F16, F16, 0, False, True, True),
    (16, 2, 128, 64, BF16, F16, 0, False, False, True),
]


@pytest.mark.parametrize(
    "heads,kv_heads,head_dim,page,io,cache,rotary,interleaved,normed,drafts", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append_norm(heads, kv_heads, head_dim, page, io, cache, rotary, interleaved, normed,
                     drafts, in_place):
    lens, new = [40, 3, 0, 129, 70], [9, 3, 2, 1, 64]
    st = Drafts(lens, new, heads, kv_heads, head_dim, page, io, cache, spare=2)
    eps = 1e-5
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    st.q[1] *= 1e-3  # rows where eps matters
    st.k[2] = 0
    w = [1 + 0.5 * torch.randn(head_dim, generator=g, device=DEV) for _ in range(2)]
    norm = kvc.HeadNorm(w[0], w[1], eps) if normed else None
    cos_sin = kvc.rope_table(140, rotary) if rotary else None
    rope = kvc.Rope(cos_sin, interleaved) if rotary else None
    before = st.pool.clone()
    q, k, v = st.q.clone(), st.k.clone(), st.v.clone()
    q_out = st.q if in_place else torch.full((st.n_tok, heads, head_dim), 7.0, dtype=io, device=DEV)
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=rope, q=st.q,
                     q_out=q_out, norm=norm, tree=st.tree if drafts else None)
    kvc.read_status(st.wsp.status, "append")
    rows, pos, slot = [], [], []
    for b, (m, n) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        d = serve_ref.depths(st.parents[b])
        s = st.slots(b)
        for i in range(n):
            rows.append(st.start[b] + i)
            pos.append(m - n + (d[i] if drafts else i))
            slot.append(int(s[m - n + i]))
    pos = torch.tensor(pos, device=DEV)
    y, bound = serve_ref.append_norm(q[rows], w[0] if normed else None, eps, cos_sin, pos,
                                     interleaved, io)
    assert bool(((q_out[rows].double() - y).abs() <= bound).all())
    y, bound = serve_ref.append_norm(k[rows], w[1] if normed else None, eps, cos_sin, pos,
                                     interleaved, cache)
    got = st.pool[1, 0, slot].double().view(y.shape)
    assert bool(((got - y).abs() <= bound).all())
    assert torch.equal(st.pool[1, 1, slot].view(v[rows].shape), v[rows].to(cache))
    # nothing else was written
    left = torch.ones(st.pool.shape[2], dtype=torch.bool, device=DEV)
    left[slot] = False
    assert torch.equal(st.pool[1][:, left].view(torch.int16), before[1][:, left].view(torch.int16))
    assert torch.equal(st.pool[0].view(torch.int16), before[0].view(torch.int16))
    others = [r for r in range(st.n_tok) if r not in rows]
    want = q[others] if in_place else torch.full_like(q[others], 7.0)
    assert torch.equal(q_out[others], want)


def test_append_norm_keys_alone_and_errors():
    st = Drafts([40, 20], [9, 5], 4, 2, 64, 16, F16, F16)
    w = torch.ones(64, device=DEV)
    norm = kvc.HeadNorm(w, w)
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, norm=norm)
    kvc.read_status(st.wsp.status, "append")
    y, bound = serve_ref.append_norm(st.k[:9], w, 1e-6, None, None, False, F16)
    got = st.pool[1, 0, st.slots(0)[31:]].double().view(y.shape)
    assert bool(((got - y).abs() <= bound).all())
    # a depth's position outside the rotation's table, and a negative one: that
    # token alone is left out
    before = st.pool.clone()
    for value in (2 ** 31 - 1, -2 ** 31, -32, 33):
        st.tree.depth[3] = value
        st.pool.copy_(before)
        kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, norm=norm,
                         rope=kvc.Rope(kvc.rope_table(64, 64)), tree=st.tree)
        assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
        st.wsp.status.zero_()
        s = st.slots(0)
        assert torch.equal(st.pool[1, :, s[34]], before[1, :, s[34]])
        assert not torch.equal(st.pool[1, 0, s[35]], before[1, 0, s[35]])


# ------------------------------------------------------------------- keep
@pytest.mark.parametrize("page,kv_heads,head_dim,layers", [(16, 2, 64, 3), (1, 1, 96, 2),
                                                            (7, 5, 128, 2), (100, 3, 256, 5)])
def test_keep(page, kv_heads, head_dim, layers):
    new = [1, 60, 33, 7, 9, 20, 5, 64]
    lens = [1, 75, 33, 300, 0, 21, 50, 190]
    paths = [[0], [0, 1, 2, 9, 10, 11, 12, 13, 14, 40, 59], [32], [], [3], list(range(20)),
             [1, 3, 4], list(range(0, 64, 2))]
    st = Setup(lens, new, kv_heads, kv_heads, head_dim, page, F16, F16, layers=layers)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    bits = st.pool.view(torch.int16)
    bits.copy_(torch.randint(-32768, 32768, bits.shape, generator=g, device=DEV).short())
    want = bits.clone()
    wide = 40
    path = torch.full((8, wide), -5, dtype=torch.int32)
    after = []
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p)
        s, base = st.slots(b), lens[b] - new[b]
        if lens[b]:
            want[:, :, s[[base + i for i in range(len(p))]]] = bits[:, :, s[[base + t for t in p]]]
        after.append(base + len(p) if lens[b] else 0)
    kept = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
    new_lens = torch.full((8,), -1, dtype=torch.int32, device=DEV)
    kvc.keep_async(st.desc, st.batch, st.pool, path.to(DEV), kept, new_lens, st.n_tok,
                   st.wsp.status)
    kvc.read_status(st.wsp.status, "keep")
    assert new_lens.tolist() == after
    assert torch.equal(bits, want)


def test_keep_errors():
    good = [0, 2, 5]
    for path, kept in (([0, 2, 2], 3), ([2, 0, 5], 3), ([0, 2, 9], 3), ([-1, 2, 5], 3),
                       (good, 4), (good, -1), ([0, 2, 2 ** 31 - 1], 3)):
        st = Setup([30, 40], [9, 9], 2, 2, 64, 16, F16, F16)
        st.pool.zero_()
        st.pool[:, :, st.slots(0)] = 1.0 + torch.arange(30, device=DEV)[:, None].half()
        st.pool[:, :, st.slots(1)] = 1.0 + torch.arange(40, device=DEV)[:, None].half()
        before = st.pool.clone()
        p = torch.tensor([path, good], dtype=torch.int32, device=DEV)
        k = torch.tensor([kept, 3], dtype=torch.int32, device=DEV)
        new_lens = torch.zeros(2, dtype=torch.int32, device=DEV)
        kvc.keep_async(st.desc, st.batch, st.pool, p, k, new_lens, 18, st.wsp.status)
        assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
        assert new_lens.tolist() == [30, 34]  # the first stays as it is, the second is kept
        s = st.slots(0)
        assert torch.equal(st.pool[:, :, s], before[:, :, s])
        s = st.slots(1)
        assert torch.equal(st.pool[:, :, s[31:34]], before[:, :, s[[31, 33, 36]]])


# ---------------------------------------------------------------- together
def test_a_step_with_drafts():
    """Append a tree, attend, keep a path; then the next tree on top.  The
    cache and the kept rows' outputs are those of a plain prompt made of the
    accepted tokens."""
    heads, kv_heads, dim, page = 8, 2, 64, 16
    st = Drafts([100, 57], [12, 9], heads, kv_heads, dim, page, F16, F16, kind="random")
    plain = Setup([100, 57], [12, 9], heads, kv_heads, dim, page, F16, F16)
    plain.pool.copy_(st.pool)
    w = 1 + 0.1 * torch.arange(dim, device=DEV).float() / dim
    norm, rope = kvc.HeadNorm(w, w), kvc.Rope(kvc.rope_table(200, dim))
    q = torch.empty((st.n_tok, heads, dim), dtype=F16, device=DEV)
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=rope, q=st.q, q_out=q,
                     norm=norm, tree=st.tree)
    out = torch.empty_like(q)
    kvc.attend_tree_async(st.desc, st.batch, st.tree, 1, st.pool, q, out, st.wsp)
    # the deepest token's path from its root
    paths = []
    for p in st.parents:
        d = serve_ref.depths(p)
        t, path = d.index(max(d)), []
        while t >= 0:
            path.append(t)
            t = p[t]
        paths.append(path[::-1])
    wide = max(len(p) for p in paths)
    path = torch.tensor([p + [0] * (wide - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    kept = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
    new_lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    kvc.keep_async(st.desc, st.batch, st.pool, path, kept, new_lens, st.n_tok, st.wsp.status)
    kvc.read_status(st.wsp.status, "drafts")
    base = [88, 48]
    assert new_lens.tolist() == [b + len(p) for b, p in zip(base, paths)]
    # the accepted tokens as a prompt
    rows = [st.start[b] + t for b, p in enumerate(paths) for t in p]
    q_start = torch.tensor([0, len(paths[0]), len(rows)], dtype=torch.int32, device=DEV)
    batch = kvc.PagedBatch(st.table, new_lens, q_start=q_start, max_len=100)
    wsp = kvc.PagedWorkspace(st.desc, batch, len(rows))
    q2 = torch.empty((len(rows), heads, dim), dtype=F16, device=DEV)
    kvc.append_async(st.desc, batch, 1, plain.pool, st.k[rows].contiguous(),
                     st.v[rows].contiguous(), wsp, rope=rope, q=st.q[rows].contiguous(), q_out=q2,
                     norm=norm)
    out2 = torch.empty_like(q2)
    kvc.attend_prompt_async(st.desc, batch, 1, plain.pool, q2, out2, wsp)
    kvc.read_status(wsp.status, "prompt")
    assert torch.equal(q2, q[rows])
    for b in range(2):
        s = st.slots(b)[: int(new_lens[b])]
        assert torch.equal(st.pool[1][:, s], plain.pool[1][:, s])
        k, v = (plain.pool[1, kv, s].view(-1, kv_heads, dim) for kv in range(2))
        a, e = int(q_start[b]), int(q_start[b + 1])
        pos = list(range(base[b], int(new_lens[b])))
        o, _, bound, _ = ref.attend(q2[a:e], k, v, pos, dim ** -0.5, 0, F16, F16, 11)
        assert bool(((out2[a:e].double() - o).abs() <= bound).all())
        assert bool(((out[rows][a:e].double() - o).abs() <= bound).all())


def test_drafts_captured_and_replayed():
    """append, attend and keep in one graph, replayed as lengths change,
    against eager calls, with the program's own work in between."""
    st = Drafts([300, 140], [20, 12], 8, 2, 64, 16, F16, F16)
    w = torch.ones(64, device=DEV)
    norm, rope = kvc.HeadNorm(w, w), kvc.Rope(kvc.rope_table(400, 64))
    path = torch.tensor([[0, 3, 7], [0, 1, 11]], dtype=torch.int32, device=DEV)
    kept = torch.tensor([3, 2], dtype=torch.int32, device=DEV)

    def step(pool, q, out, new_lens, wsp, stream=None):
        kvc.tree_async(st.desc, st.batch, st.tree, wsp)
        kvc.append_async(st.desc, st.batch, 1, pool, st.k, st.v, wsp, rope=rope, q=st.q, q_out=q,
                         norm=norm, tree=st.tree)
        kvc.attend_tree_async(st.desc, st.batch, st.tree, 1, pool, q, out, wsp)
        kvc.keep_async(st.desc, st.batch, pool, path, kept, new_lens, st.n_tok, wsp.status)

    def buffers():
        return (st.pool.clone(), torch.zeros_like(st.q),
                torch.zeros(st.q.shape, dtype=F16, device=DEV),
                torch.zeros(2, dtype=torch.int32, device=DEV),
                kvc.PagedWorkspace(st.desc, st.batch, st.n_tok, tree=st.tree))

    mine, want = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(*mine)
        with torch.cuda.graph(graph, stream=side):
            step(*mine)
    torch.cuda.current_stream().wait_stream(side)
    for lens in ([300, 140], [21, 12], [260, 0], [300, 77]):
        st.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for bufs in (mine, want):
            bufs[0].copy_(st.pool)
            for t in bufs[1:4]:
                t.zero_()
        graph.replay()
        step(*want)
        torch.cuda.synchronize()
        for a, b in zip(mine[:4], want[:4]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert bool((mine[2] != 0).any())
    kvc.read_status(mine[4].status, "graph")


def test_drafts_on_another_stream():
    """Every call on a stream of its own, against the current stream's."""
    st = Drafts([700, 90], [20, 12], 8, 2, 64, 16, F16, F16)
    w = torch.ones(64, device=DEV)
    norm, rope = kvc.HeadNorm(w, w), kvc.Rope(kvc.rope_table(800, 64))
    path = torch.tensor([[0, 3, 7], [0, 1, 11]], dtype=torch.int32, device=DEV)
    kept = torch.tensor([3, 2], dtype=torch.int32, device=DEV)
    results = []
    for stream in (None, torch.cuda.Stream()):
        pool, q = st.pool.clone(), torch.zeros(st.q.shape, dtype=F16, device=DEV)
        out = torch.zeros_like(q)
        new_lens = torch.zeros(2, dtype=torch.int32, device=DEV)
        tree = kvc.Tree(st.tree.parent, 20)
        wsp = kvc.PagedWorkspace(st.desc, st.batch, st.n_tok, tree=tree)
        kvc.tree_async(st.desc, st.batch, tree, wsp, stream=stream)
        kvc.append_async(st.desc, st.batch, 1, pool, st.k, st.v, wsp, rope=rope, q=st.q, q_out=q,
                         norm=norm, tree=tree, stream=stream)
        kvc.attend_tree_async(st.desc, st.batch, tree, 1, pool, q, out, wsp, stream=stream)
        kvc.keep_async(st.desc, st.batch, pool, path, kept, new_lens, st.n_tok, wsp.status,
                       stream=stream)
        kvc.read_status(wsp.status, "drafts", stream)
        results.append((pool.view(torch.int16), q, out, new_lens))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert bool((results[0][2] != 0).any())
