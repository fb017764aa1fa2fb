"""The paged-cache operators on the GPU against plain 64-bit forms: appending
with rotation, attention of one and of several new tokens, page moves, and
the codec's restore feeding them.  Unused slots of every pool hold NaN and
infinities."""
import ctypes

import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
F16, BF16 = torch.float16, torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Setup:
    """A pool of two layers with scattered pages for sequences of these
    lengths; what no token uses holds NaN and infinities."""

    def __init__(self, lens, new, heads, kv_heads, head_dim, page, io, cache, seed=1,
                 spare=0, single=False, layers=2):
        g = _gen(seed)
        self.lens_host, self.new_host, self.page = list(lens), list(new), page
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.io, self.cache = io, cache
        need = [(m + page - 1) // page for m in lens]
        self.n_pages = sum(need) + 3
        ids = torch.randperm(self.n_pages, generator=g, device=DEV).tolist()
        width = max(need + [1])
        rows, at = [], 0
        for n in need:
            # entries behind the last page are never read: ids far outside
            rows.append(ids[at:at + n] + [-(2 ** 31)] * (width - n))
            at += n
        self.table = torch.tensor(rows, dtype=torch.int32, device=DEV).view(len(lens), width)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        self.start = start
        self.n_tok = start[-1] + spare
        self.desc = kvc.make_paged_desc(layers, heads, kv_heads, head_dim, page, self.n_pages,
                                        cache_dtype=cache, io_dtype=io)
        q_start = None if single else torch.tensor(start, dtype=torch.int32, device=DEV)
        self.batch = kvc.PagedBatch(self.table, self.lens, q_start=q_start,
                                    max_len=max(max(lens), 1))
        self.wsp = kvc.PagedWorkspace(self.desc, self.batch, self.n_tok)
        c = kv_heads * head_dim
        self.pool = torch.empty(self.desc.pool_shape, dtype=cache, device=DEV)
        self.pool.fill_(float("nan"))
        self.pool[:, :, ::3] = float("inf")
        for b, m in enumerate(lens):
            s = self.slots(b)
            for kv in range(2):
                x = torch.randn((m, c), generator=g, device=DEV)
                self.pool[1, kv, s] = (x * (1.0 + 0.5 * kv) + 0.3).to(cache)
        # q, k and v as slices of one projection's rows
        w = (heads + 2 * kv_heads) * head_dim
        qkv = torch.randn((self.n_tok, w), generator=g, device=DEV).to(io)
        self.q = qkv[:, : heads * head_dim].unflatten(1, (heads, head_dim))
        self.k = qkv[:, heads * head_dim: (heads + kv_heads) * head_dim].unflatten(
            1, (kv_heads, head_dim))
        self.v = qkv[:, (heads + kv_heads) * head_dim:].unflatten(1, (kv_heads, head_dim))

    def slots(self, b):
        return ref.slots(self.table[b], self.lens_host[b], self.page, DEV)

    def cached(self, b, layer=1):
        s = self.slots(b)
        shape = (-1, self.kv_heads, self.head_dim)
        return self.pool[layer, 0, s].view(shape), self.pool[layer, 1, s].view(shape)


def _attend(st, window=0, scale=None, prompt=False, stream=None):
    out = torch.full((st.n_tok, st.heads, st.head_dim), 7.0, dtype=st.io, device=DEV)
    lse = torch.full((st.n_tok, st.heads), 7.0, device=DEV)
    f = kvc.attend_prompt_async if prompt else kvc.attend_async
    f(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, scale=scale, window=window, lse=lse,
      stream=stream)
    kvc.read_status(st.wsp.status, "attend", stream)
    return out, lse


def _check_attend(st, out, lse, window=0, scale=None):
    scale = st.head_dim ** -0.5 if scale is None else scale
    for b, (m, n) in enumerate(zip(st.lens_host, st.new_host)):
        a = st.start[b]
        k, v = st.cached(b)
        pos = list(range(m - n, m))
        o, e, bo, be = ref.attend(st.q[a:a + n], k, v, pos, scale, window, st.cache, st.io)
        got, got_e = out[a:a + n].double(), lse[a:a + n].double()
        empty = torch.isinf(e)
        assert torch.equal(got_e[empty], e[empty])
        assert bool((got[empty] == 0).all())
        full = ~empty  # empty rows were compared above: zeros, bound zero
        worst = ((got - o).abs() / bo)[full].max().item() if bool(full.any()) else 0.0
        worst_e = ((got_e - e).abs() / be)[full].max().item() if bool(full.any()) else 0.0
        assert worst <= 1.0 and worst_e <= 1.0, (b, m, n, worst, worst_e)
        assert bool(torch.isfinite(got).all())
    a = st.start[-1]
    assert bool((out[a:] == 7.0).all()) and bool((lse[a:] == 7.0).all())


SINGLE = [
    # heads, kv_heads, head_dim, page, io, cache, lens, window
    (8, 2, 64, 16, F16, F16, [1, 2, 15, 16, 17, 31, 32, 33], 0),
    (4, 4, 128, 16, BF16, BF16, [127, 128, 129, 0, 1, 513], 0),
    (64, 8, 128, 16, F16, F16, [1500], 0),
    (64, 8, 128, 64, BF16, F16, [3001, 7], 0),
    (14, 2, 96, 20, F16, F16, [100, 0, 257, 40], 33),
    (40, 1, 128, 1, BF16, BF16, [300, 65], 0),
    (6, 2, 256, 48, BF16, F16, [700, 3, 64], 0),
    (5, 5, 256, 7, F16, F16, [90, 301], 1),
    (128, 1, 64, 1500, F16, F16, [1499, 1500, 1501], 1000),
    (17, 1, 64, 8, BF16, BF16, [0, 0, 5], 4),
    # more sequences than a search step takes, cut at arbitrary places, and not cut
    (4, 1, 64, 16, F16, F16, [(i * 37) % 23 * 30 + i % 5 for i in range(300)], 0),
    (6, 3, 64, 10, BF16, BF16, [(i * 13) % 29 * 17 for i in range(520)], 0),
    (3, 1, 96, 16, F16, F16, [2000] + [0] * 260 + [1500, 1, 600], 900),
    (20, 1, 128, 16, BF16, F16, [1100, 513, 2300], 0),
    # two and four KV heads side by side, groups that pass a row tile
    (12, 6, 64, 16, F16, F16, [700, 33, 1025, 0, 2], 0),
    (68, 4, 96, 7, BF16, BF16, [640, 800, 31], 500),
    (8, 8, 256, 16, F16, F16, [900, 513], 0),
    # more than 16 heads to a KV head over long caches and short ones
    (66, 2, 128, 16, BF16, BF16, [700, 0, 1, 65, 1300], 0),
    (128, 1, 256, 10, F16, F16, [600, 90], 130),
    (40, 2, 96, 16, BF16, F16, [400, 1, 0, 33], 60),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,window", SINGLE)
def test_attend_single(heads, kv_heads, head_dim, page, io, cache, lens, window):
    st = Setup(lens, [1] * len(lens), heads, kv_heads, head_dim, page, io, cache, single=True)
    out, lse = _attend(st, window)
    _check_attend(st, out, lse, window)


PROMPT = [
    # heads, kv_heads, head_dim, page, io, cache, lens, new, window
    (8, 2, 64, 16, F16, F16, [5, 40, 33], [5, 3, 33], 0),
    (4, 4, 128, 16, BF16, BF16, [130, 1, 200], [130, 1, 129], 0),
    (16, 2, 128, 16, BF16, F16, [600, 64, 311], [37, 64, 300], 0),
    (14, 2, 96, 20, F16, F16, [150, 300], [150, 41], 50),
    (11, 1, 256, 10, BF16, BF16, [90, 257], [90, 20], 0),
    (3, 3, 256, 64, F16, F16, [200], [131], 1),
    (6, 6, 64, 1, F16, F16, [70, 3, 65], [70, 0, 64], 7),
    (64, 1, 64, 32, BF16, F16, [129], [9], 0),
    # a few tokens over long caches, split, beside sequences without new tokens
    (8, 2, 64, 16, F16, F16, [900, 1500, 30, 700, 5], [9, 3, 30, 0, 1], 0),
    (6, 1, 128, 20, BF16, BF16, [1201, 33, 0, 640], [17, 5, 0, 2], 300),
    (40, 2, 256, 16, BF16, F16, [800, 513], [3, 2], 0),
    (4, 4, 128, 16, BF16, F16, [1300, 700, 90], [20, 3, 40], 0),
    # 128-row tiles: a split context, no grouping, a group of 7 and of 128, windows
    (8, 2, 128, 16, F16, F16, [2050], [40], 0),
    (2, 2, 128, 64, BF16, BF16, [257, 700], [257, 129], 0),
    (7, 1, 128, 20, BF16, F16, [333, 0, 90], [333, 0, 3], 100),
    (128, 1, 64, 16, F16, F16, [70, 5], [3, 5], 0),
    (8, 1, 96, 48, BF16, BF16, [1300], [33], 700),
    (4, 1, 256, 16, F16, F16, [530], [64], 0),
    (6, 2, 64, 7, F16, F16, [64, 128, 127], [64, 64, 127], 65),
    # a long prompt beside single tokens, and many of a few tokens
    (8, 1, 64, 16, F16, F16, [300] + [70 + 9 * i for i in range(40)], [140] + [1] * 40, 0),
    (8, 2, 64, 16, BF16, F16, [50 + 11 * i for i in range(70)], [4] * 70, 0),
    # 256-row tiles: causal from the first token, a window, a split context, odd pages
    (16, 1, 64, 16, F16, F16, [130, 200, 77], [130, 64, 77], 0),
    (32, 2, 128, 20, BF16, BF16, [300], [75], 130),
    (24, 1, 96, 7, BF16, F16, [1500], [44], 0),
    (128, 1, 128, 16, F16, F16, [65, 9], [9, 9], 0),
    (1, 1, 128, 64, BF16, BF16, [1100], [1100], 100),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,new,window", PROMPT)
def test_attend_prompt(heads, kv_heads, head_dim, page, io, cache, lens, new, window):
    st = Setup(lens, new, heads, kv_heads, head_dim, page, io, cache, spare=3)
    out, lse = _attend(st, window, prompt=True)
    _check_attend(st, out, lse, window)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_attend_scales(scale):
    """A scale of any sign: at 3 a row's weight lies on one token or two."""
    st = Setup([200, 40], [1, 1], 8, 2, 128, 16, F16, F16, single=True)
    out, lse = _attend(st, scale=scale)
    _check_attend(st, out, lse, scale=scale)


def test_attend_padding_rows():
    """More new tokens than the sequence holds: the rows of negative position
    are padding and come back as zeros; lengths of zero and no sequences."""
    st = Setup([3, 0, 40], [7, 5, 2], 8, 2, 64, 16, F16, F16, spare=2)
    out, lse = _attend(st, prompt=True)
    _check_attend(st, out, lse)


@pytest.mark.parametrize("heads", [2, 8, 40])  # 128 (partly and well filled) and 256 rows a workgroup
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attend_nonfinite_hidden_values(dtype, heads):
    """Infinities and NaN in the cached rows of tokens that a row does not
    see (later tokens of the same prompt, tokens before its window) have no
    effect on that row."""
    st = Setup([90, 64], [60, 64], heads, 2, 64, 16, dtype, dtype, spare=1)
    window = 24
    bad = [(0, 80), (0, 45), (1, 63), (1, 20)]
    for b, t in bad:
        s = int(st.slots(b)[t])
        st.pool[1, 0, s] = float("nan")
        st.pool[1, 1, s, ::2] = float("inf")
        st.pool[1, 1, s, 1::2] = float("nan")
    out, lse = _attend(st, window, prompt=True)
    for b in range(2):
        m, n, a = st.lens_host[b], st.new_host[b], st.start[b]
        k, v = st.cached(b)
        k, v = k.clone(), v.clone()
        hit = [t for c, t in bad if c == b]
        k[hit], v[hit] = 0.0, 0.0  # rows that see one of them are skipped below
        o, e, bo, be = ref.attend(st.q[a:a + n], k, v, list(range(m - n, m)), 64 ** -0.5, window,
                                  dtype, dtype)
        clean = 0
        for i in range(n):
            p = m - n + i
            if any(p - window < t <= p for t in hit):
                assert bool(torch.isnan(out[a + i]).all())
                continue
            clean += 1
            assert bool(((out[a + i].double() - o[i]).abs() <= bo[i]).all()), (b, i)
            assert bool(((lse[a + i].double() - e[i]).abs() <= be[i]).all()), (b, i)
        assert clean > 3


def test_attend_long_tail_of_small_probabilities():
    """One token far above thousands of others whose weights, each below half
    a binary16 step of the largest, together make up a tenth of the sum."""
    m, d = 4097, 64
    st = Setup([m], [1], 1, 1, d, 16, F16, F16, single=True)
    s = st.slots(0)
    st.pool[1, 0, s] = 0.0
    st.pool[1, 0, s[100], 0] = 1.0
    st.pool[1, 1, s] = 1.0
    st.pool[1, 1, s[100]] = 0.0
    st.q.zero_()
    st.q[0, 0, 0] = 8.0
    scale = 1.3  # exp(-10.4) = 2^-15
    out, lse = _attend(st, scale=scale)
    _check_attend(st, out, lse, scale=scale)
    st.q[0, 0, 0] = 16.0  # exp(-20.8) = 2^-30: 4,096 of them are 2^-18
    out, lse = _attend(st, scale=scale)
    _check_attend(st, out, lse, scale=scale)
    assert out.abs().min().item() > 0


APPEND = [
    # heads, kv_heads, head_dim, page, io, cache, lens, new, rotary, interleaved
    (64, 8, 128, 16, F16, F16, [9, 1, 700], None, 128, False),
    (8, 8, 64, 16, BF16, BF16, [64, 33], [64, 20], 64, True),
    (4, 2, 96, 20, BF16, F16, [50, 3, 21], [50, 0, 21], 48, False),
    (4, 2, 96, 1, F16, F16, [50, 3, 21], [1, 2, 3], 32, True),
    (9, 3, 256, 7, BF16, F16, [30], [30], 16, False),
    (2, 1, 64, 1500, F16, F16, [1600], [1503], 0, False),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,new,rotary,inter", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append(heads, kv_heads, head_dim, page, io, cache, lens, new, rotary, inter, in_place):
    single = new is None
    new = [1] * len(lens) if single else new
    st = Setup(lens, new, heads, kv_heads, head_dim, page, io, cache, single=single,
               spare=0 if single else 2)
    rope = None
    if rotary:
        rope = kvc.Rope(kvc.rope_table(max(lens), rotary, device=DEV), interleaved=inter)
    q0, pool0 = st.q.clone(), st.pool.clone()
    q_out = st.q if in_place else torch.full_like(st.q.contiguous(), 7.0)
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=rope, q=st.q,
                     q_out=q_out)
    kvc.read_status(st.wsp.status, "append")
    written = torch.zeros(st.pool.shape[2], dtype=torch.bool, device=DEV)
    for b, (m, n) in enumerate(zip(lens, new)):
        a, pos = st.start[b], torch.arange(m - n, m, device=DEV)
        s = st.slots(b)[m - n:]
        written[s] = True
        k, v = st.k[a:a + n].double(), st.v[a:a + n]
        q = q0[a:a + n].double()
        got_k = st.pool[1, 0, s].view(n, kv_heads, head_dim)
        got_v = st.pool[1, 1, s].view(n, kv_heads, head_dim)
        assert torch.equal(got_v, v.to(cache))
        if rope is None:
            assert torch.equal(got_k, st.k[a:a + n].to(cache))
            assert torch.equal(q_out[a:a + n], q0[a:a + n])
            continue
        y, mag = ref.rotate(k, rope.cos_sin, pos, inter)
        assert bool(((got_k.double() - y).abs() <= ref.rotate_bound(y, mag, cache)).all())
        y, mag = ref.rotate(q, rope.cos_sin, pos, inter)
        assert bool(((q_out[a:a + n].double() - y).abs() <= ref.rotate_bound(y, mag, io)).all())
    # nothing else was touched: other slots, the other layer, rows behind the last sequence
    def bits(x):
        return x.view(torch.int16)
    assert torch.equal(bits(st.pool[0]), bits(pool0[0]))
    assert torch.equal(bits(st.pool[1][:, ~written]), bits(pool0[1][:, ~written]))
    a = st.start[-1]
    assert torch.equal(q_out[a:], q0[a:] if in_place else torch.full_like(q_out[a:], 7.0))


@pytest.mark.parametrize("inter", [False, True])
def test_append_beyond_the_caches(inter):
    """A call that moves more than 256 MB (287 MB here) goes past the caches:
    the same bits as the same tokens in calls of a third."""
    n = 7002
    st = Setup([n + 5], [n], 64, 8, 128, 16, BF16, F16, layers=2)
    rope = kvc.Rope(kvc.rope_table(n + 5, 128, device=DEV), interleaved=inter)
    q_out = torch.zeros_like(st.q.contiguous())
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=rope, q=st.q,
                     q_out=q_out)
    kvc.read_status(st.wsp.status, "append")
    pool, q2 = st.pool.clone(), torch.zeros_like(q_out)
    pool[1][:, st.slots(0)[5:]] = 0
    for a in range(0, n, n // 3):
        rows = slice(a, a + n // 3)
        st.lens.fill_(5 + a + n // 3)
        part = kvc.PagedBatch(st.table, st.lens, max_len=n + 5,
                              q_start=torch.tensor([0, n // 3], dtype=torch.int32, device=DEV))
        kvc.append_async(st.desc, part, 1, pool, st.k[rows], st.v[rows], st.wsp, rope=rope,
                         q=st.q[rows], q_out=q2[rows])
    kvc.read_status(st.wsp.status, "append")
    assert torch.equal(pool.view(torch.int16), st.pool.view(torch.int16))
    assert torch.equal(q2, q_out)


def test_page_moves_beyond_the_caches():
    layers, n, page, c = 9, 4001, 20, 1024  # 295 MB read and written
    g = _gen(8)
    n_pages = 210
    desc = kvc.make_paged_desc(layers, 8, 8, 128, page, n_pages)
    pool = torch.randn(desc.pool_shape, generator=g, device=DEV).to(F16)
    table = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s = ref.slots(table, n + 3, page, DEV)[3:]
    flat = torch.zeros((layers, 2, n + 1, c), dtype=F16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvc.page_out_async(desc, pool, table, 3, n, flat, 1, status)
    assert torch.equal(flat[:, :, 1:], pool[:, :, s]) and bool((flat[:, :, 0] == 0).all())
    flat.neg_()
    want = pool.clone()
    want[:, :, s] = flat[:, :, 1:]
    kvc.page_in_async(desc, flat, 1, pool, table, 3, n, status)
    assert torch.equal(pool, want)
    kvc.read_status(status, "pages")


def test_append_padding_and_keys_only():
    """Rows of negative position are skipped; q may be left out."""
    st = Setup([0, 5, 0], [1, 1, 1], 4, 2, 64, 16, F16, F16, single=True)
    pool0 = st.pool.clone()
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
    kvc.read_status(st.wsp.status, "append")
    s = int(st.slots(1)[4])
    assert torch.equal(st.pool[1, 0, s], st.k[1].flatten())
    pool0[1, 0, s], pool0[1, 1, s] = st.k[1].flatten(), st.v[1].flatten()
    assert torch.equal(st.pool.view(torch.int16), pool0.view(torch.int16))
    q_out = torch.full_like(st.q.contiguous(), 7.0)
    rope = kvc.Rope(kvc.rope_table(5, 64, device=DEV))
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=rope, q=st.q,
                     q_out=q_out)
    kvc.read_status(st.wsp.status, "append")
    assert bool((q_out[[0, 2]] == 7.0).all()) and not bool((q_out[1] == 7.0).any())


def test_append_overflow_to_binary16():
    """A bfloat16 value beyond binary16's range is stored as an infinity."""
    st = Setup([1], [1], 1, 1, 64, 16, BF16, F16, single=True)
    st.v.fill_(7e4)
    st.v[0, 0, 0] = -1e38
    st.v[0, 0, 1] = 65000.0
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
    got = st.pool[1, 1, int(st.slots(0)[0])]
    assert got[0].item() == float("-inf") and bool((got[2:] == float("inf")).all())
    assert got[1].item() == 65024.0


@pytest.mark.parametrize("page,kv_heads,head_dim,first,n,extra", [
    (16, 4, 128, 0, 1500, 0), (16, 8, 128, 5, 40, 3), (20, 1, 64, 19, 2, 1),
    (1, 3, 96, 0, 33, 0), (1500, 2, 256, 1400, 300, 9), (7, 5, 64, 3, 1, 4)])
def test_page_moves(page, kv_heads, head_dim, first, n, extra):
    st = Setup([first + n], [1], kv_heads, kv_heads, head_dim, page, F16, F16, single=True,
               layers=3)
    g = _gen(5)
    c = kv_heads * head_dim
    st.pool.copy_(torch.randn(st.pool.shape, generator=g, device=DEV).to(F16))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    flat = torch.full((3, 2, n + extra, c), 7.0, dtype=F16, device=DEV)
    kvc.page_out_async(st.desc, st.pool, st.table[0], first, n, flat, extra // 2, status)
    s = st.slots(0)[first:]
    want = torch.full_like(flat, 7.0)
    want[:, :, extra // 2: extra // 2 + n] = st.pool[:, :, s]
    kvc.read_status(status, "page_out")
    assert torch.equal(flat, want)
    src = torch.randn(flat.shape, generator=g, device=DEV).to(F16)
    pool = st.pool.clone()
    pool[:, :, s] = src[:, :, extra // 2: extra // 2 + n]
    kvc.page_in_async(st.desc, src, extra // 2, st.pool, st.table[0], first, n, status)
    kvc.read_status(status, "page_in")
    assert torch.equal(st.pool, pool)


def test_device_errors_are_reported():
    """Bad page ids, lengths, positions and q_start: KVC_ERR_SHAPE in the
    status word, which the calls do not clear."""
    def code(st):
        c = int(st.wsp.status.item())
        st.wsp.status.zero_()
        return c

    for bad in (-1, 10 ** 6, -(2 ** 31)):
        st = Setup([40, 50], [1, 1], 4, 2, 64, 16, F16, F16, single=True)
        st.table[1, 2] = bad  # tokens 32..47 of the second sequence
        _kw = dict(rope=None)
        out = torch.zeros((2, 4, 64), dtype=F16, device=DEV)
        kvc.attend_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
        assert code(st) == kvc.ERR_SHAPE
        st.lens[1] = 41
        pool0 = st.pool.clone()
        kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, **_kw)
        assert code(st) == kvc.ERR_SHAPE
        s0 = int(st.slots(0)[39])
        pool0[1, 0, s0], pool0[1, 1, s0] = st.k[0].flatten(), st.v[0].flatten()
        assert torch.equal(st.pool.view(torch.int16), pool0.view(torch.int16))
        flat = torch.zeros((2, 2, 50, 128), dtype=F16, device=DEV)
        kvc.page_out_async(st.desc, st.pool, st.table[1], 0, 50, flat, 0, st.wsp.status)
        assert code(st) == kvc.ERR_SHAPE
        kvc.page_in_async(st.desc, flat, 0, st.pool, st.table[1], 0, 50, st.wsp.status)
        assert code(st) == kvc.ERR_SHAPE
    st = Setup([40, 50], [1, 1], 4, 2, 64, 16, F16, F16, single=True)
    for bad in (51, 2 ** 31 - 1, -1):
        st.lens[0] = bad
        kvc.attend_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
        assert code(st) == kvc.ERR_SHAPE
        kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
        assert code(st) == kvc.ERR_SHAPE
    st.lens[0] = 40
    short = kvc.Rope(kvc.rope_table(49, 64, device=DEV))  # position 49 is missing
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, rope=short)
    assert code(st) == kvc.ERR_SHAPE
    st = Setup([40, 50], [20, 10], 4, 2, 64, 16, F16, F16)
    out = torch.zeros((30, 4, 64), dtype=F16, device=DEV)
    for bad in ([0, 20, 31], [0, -1, 30], [5, 4, 30], [0, 2 ** 31 - 1, 30]):
        st.batch.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        kvc.attend_prompt_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
        assert code(st) == kvc.ERR_SHAPE
        kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
        assert code(st) == kvc.ERR_SHAPE


@pytest.mark.parametrize("heads", [2, 64])  # 128 rows a workgroup
def test_q_start_that_overlaps_itself(heads):
    """Every other sequence claims all rows: reported, and the call ends."""
    n = 600
    st = Setup([40] * n, [1] * n, heads, 1, 64, 16, F16, F16)
    st.batch.q_start[0::2] = 0
    st.batch.q_start[1::2] = n
    out = torch.zeros((n, heads, 64), dtype=F16, device=DEV)
    kvc.attend_prompt_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
    assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
    st.wsp.status.zero_()
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
    assert int(st.wsp.status.item()) == kvc.ERR_SHAPE


def test_binding_refuses_what_it_cannot_pass_on(monkeypatch):
    st = Setup([40], [1], 4, 2, 64, 16, F16, F16, single=True)
    out = torch.empty_like(st.q.contiguous())
    flat = torch.zeros((2, 2, 50, 128), dtype=F16, device=DEV)

    def attend(**kw):
        a = dict(layer=1, pool=st.pool, q=st.q, out=out, window=0, lse=None)
        a.update(kw)
        kvc.attend_async(st.desc, st.batch, a["layer"], a["pool"], a["q"], a["out"], st.wsp,
                         window=a["window"], lse=a["lse"])

    for bad in (dict(layer=-1), dict(layer=1 << 32), dict(window=-1), dict(window=1 << 32),
                dict(pool=st.pool[:1]), dict(pool=st.pool.to(BF16)), dict(q=st.q.to(BF16)),
                dict(q=st.q.cpu()), dict(q=st.q.transpose(1, 2)), dict(out=out[:, :2]),
                dict(lse=torch.zeros((1, 3), device=DEV)),
                dict(lse=torch.zeros((1, 4), dtype=torch.float64, device=DEV))):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(kvc.KvcError):
        attend(layer=2)
    for first, n, at in ((1 << 32, 1, 0), (0, -1, 0), (0, 1, 1 << 32)):
        with pytest.raises(ValueError):
            kvc.page_out_async(st.desc, st.pool, st.table[0], first, n, flat, at, st.wsp.status)
    with pytest.raises(ValueError):
        kvc.PagedBatch(st.table, st.lens, max_len=1 << 32)
    with pytest.raises(ValueError):
        kvc.PagedBatch(st.table, st.lens.to(torch.int64))
    with pytest.raises(ValueError):
        kvc.make_paged_desc(1, 8, 2, 64 + (1 << 32), 16, 4)
    with monkeypatch.context() as m:  # as on a box where another device is current
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError):
            attend()
    small = kvc.PagedWorkspace(st.desc, st.batch)
    long = kvc.PagedBatch(torch.zeros((1, 4), dtype=torch.int32, device=DEV), st.lens, max_len=64)
    attend()  # and a good call still goes through, on a pool of bit patterns too
    assert int(st.wsp.status.item()) == 0
    want = out.clone()
    attend(pool=st.pool.view(torch.int16))
    assert torch.equal(out, want)
    q = st.q.clone()
    attend(q=q, out=q)  # the queries' own place
    assert torch.equal(q, want)
    big = kvc.make_paged_desc(2, 4, 2, 64, 1 << 20, 4)
    pool = torch.zeros((1,), dtype=F16, device=DEV)
    with pytest.raises(ValueError):
        kvc.attend_async(big, long, 1, pool, st.q, out, small)
    table = torch.zeros((1, 400), dtype=torch.int32, device=DEV)
    wide = kvc.PagedBatch(table, st.lens)
    with pytest.raises(kvc.KvcError) as e:  # a longer cache needs more scratch
        kvc.attend_async(st.desc, wide, 1, st.pool, st.q, out, small)
    assert e.value.code == kvc.ERR_CAPACITY


def test_status_word_is_sticky():
    st = Setup([40], [1], 4, 2, 64, 16, F16, F16, single=True)
    st.wsp.status.fill_(-5)
    out = torch.zeros((1, 4, 64), dtype=F16, device=DEV)
    kvc.attend_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
    assert int(st.wsp.status.item()) == -5


def test_repeated_calls_give_the_same_bits():
    st = Setup([3001, 64, 900], [1, 1, 1], 16, 2, 128, 16, F16, F16, single=True)
    first = _attend(st)
    for _ in range(5):
        st.wsp.ws.fill_(0xFF)
        again = _attend(st)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_slots_past_32_bits():
    """A pool whose last pages lie more than 2^32 elements behind the first."""
    heads, d, page = 4, 256, 64
    n_pages = (2 ** 32 // (heads * d)) // page + 40  # 4.3 G elements a plane, 17 GB in all
    st = Setup([300], [1], heads, heads, d, page, F16, F16, single=True)
    desc = kvc.make_paged_desc(1, heads, heads, d, page, n_pages)
    pool = torch.empty(desc.pool_shape, dtype=F16, device=DEV)
    table = torch.arange(n_pages - 5, n_pages, dtype=torch.int32, device=DEV)[None].contiguous()
    s = ref.slots(table[0], 300, page, DEV)
    pool[0, 0, s], pool[0, 1, s] = st.pool[1, 0, st.slots(0)], st.pool[1, 1, st.slots(0)]
    batch = kvc.PagedBatch(table, st.lens, max_len=300)
    wsp = kvc.PagedWorkspace(desc, batch)
    kvc.append_async(desc, batch, 0, pool, st.k, st.v, wsp)
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp)
    want, want_e = _attend(st)
    out, lse = torch.empty_like(want), torch.empty_like(want_e)
    kvc.attend_async(desc, batch, 0, pool, st.q, out, wsp, lse=lse)
    kvc.read_status(wsp.status, "attend")
    assert torch.equal(out, want) and torch.equal(lse, want_e)
    flat = torch.empty((1, 2, 300, heads * d), dtype=F16, device=DEV)
    kvc.page_out_async(desc, pool, table[0], 0, 300, flat, 0, wsp.status)
    assert torch.equal(flat[0], pool[0][:, s])


def test_side_stream_and_two_at_once():
    """Calls on a side stream wait for the current stream's work; two batches
    on two streams with workspaces of their own do not disturb each other."""
    a = Setup([3001, 900], [1, 1], 16, 2, 128, 16, F16, F16, single=True, seed=2)
    b = Setup([2000, 1500], [1, 1], 16, 2, 128, 16, F16, F16, single=True, seed=3)
    want_a, want_b = _attend(a), _attend(b)
    s1, s2 = torch.cuda.Stream(device=DEV), torch.cuda.Stream(device=DEV)
    x = torch.full((4096, 4096), 1e-3, device=DEV)
    for _ in range(6):
        x = x @ x
    got = []
    for st, s in ((a, s1), (b, s2)):
        out = torch.empty_like(want_a[0])
        lse = torch.empty_like(want_a[1])
        kvc.attend_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, lse=lse, stream=s)
        got.append((out, lse))
    torch.cuda.synchronize()
    for g, w in zip(got, (want_a, want_b)):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_captured_step_replayed():
    """A decode step (append, then attention) captured once and replayed while
    the lengths grow, with eager work between, against eager calls."""
    heads, kv_heads, d, page = 16, 2, 128, 16
    st = Setup([600, 0, 33], [1, 1, 1], heads, kv_heads, d, page, BF16, F16, single=True)
    # room for growth: wider tables over more pages
    n_pages, width = 120, 45
    desc = kvc.make_paged_desc(1, heads, kv_heads, d, page, n_pages, F16, BF16)
    table = torch.randperm(n_pages, generator=_gen(4), device=DEV).to(torch.int32)[: 2 * width]
    table = torch.cat([table[:width], table[width:], table[:width]]).view(3, width).contiguous()
    table[2] = torch.flip(table[1], [0])
    lens = torch.tensor([600, 0, 0], dtype=torch.int32, device=DEV)
    pool = torch.randn(desc.pool_shape, generator=_gen(6), device=DEV).to(F16)
    batch = kvc.PagedBatch(table, lens)
    wsp = kvc.PagedWorkspace(desc, batch)
    rope = kvc.Rope(kvc.rope_table(width * page, d, device=DEV))
    q, k, v = st.q.clone(), st.k.clone(), st.v.clone()
    q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros((3, heads), device=DEV)

    def step(pool, q_rot, out, lse, wsp):
        kvc.append_async(desc, batch, 0, pool, k, v, wsp, rope=rope, q=q, q_out=q_rot)
        kvc.attend_async(desc, batch, 0, pool, q_rot, out, wsp, lse=lse)

    pool2 = pool.clone()
    warm = torch.cuda.Stream(device=DEV)
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(pool2, q_rot.clone(), out.clone(), lse.clone(), wsp)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, q_rot, out, lse, wsp)
    pool2 = pool.clone()
    wsp2 = kvc.PagedWorkspace(desc, batch)
    for i in range(6):
        q.normal_(generator=_gen(10 + i))
        k.normal_(generator=_gen(20 + i))
        lens[0] += 13
        if i >= 2:
            lens[1] += 5
        r2, o2, l2 = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(lse)
        step(pool2, r2, o2, l2, wsp2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        live = lens > 0
        assert torch.equal(q_rot[live], r2[live])
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert torch.equal(pool, pool2)
    kvc.read_status(wsp.status, "step")


def test_empty_batches():
    desc = kvc.make_paged_desc(1, 4, 2, 64, 16, 4)
    table = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    lens = torch.zeros(0, dtype=torch.int32, device=DEV)
    pool = torch.zeros(desc.pool_shape, dtype=F16, device=DEV)
    for q_start in (None, torch.zeros(1, dtype=torch.int32, device=DEV)):
        batch = kvc.PagedBatch(table, lens, q_start=q_start)
        wsp = kvc.PagedWorkspace(desc, batch)
        q = torch.zeros((0, 4, 64), dtype=F16, device=DEV)
        k = torch.zeros((0, 2, 64), dtype=F16, device=DEV)
        kvc.append_async(desc, batch, 0, pool, k, k, wsp, q=q, q_out=q.clone())
        f = kvc.attend_async if q_start is None else kvc.attend_prompt_async
        f(desc, batch, 0, pool, q, q.clone(), wsp)
        kvc.read_status(wsp.status, "empty")
    flat = torch.zeros((1, 2, 0, 128), dtype=F16, device=DEV)
    t = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvc.page_out_async(desc, pool, t, 3, 0, flat, 0, wsp.status)
    kvc.page_in_async(desc, flat, 0, pool, t, 16, 0, wsp.status)
    kvc.read_status(wsp.status, "empty")


def test_context_restored_extended_and_evicted():
    """The operators as they are used together: a context's containers are
    decoded straight into consecutive pages of a pool and, for a second copy,
    into a tensor that page_in scatters; a question's tokens are appended and
    attended, then single tokens; both copies agree with the 64-bit form and,
    each called by itself, bit for bit; page_out hands the context back and encode accepts it, its
    containers equal to those of the same tokens in a tensor of their own."""
    L, hk, d, heads, page, T = 2, 2, 64, 8, 16, 3100
    g = _gen(9)
    c = hk * d
    cd = kvc.make_desc(L, c, [(6, 5, 4), (5, 4, 3)])
    kv = (torch.randn((L, 2, T, c), generator=g, device=DEV) + 0.5).to(F16)
    prof = (torch.randn((L, 2, 1500, c), generator=g, device=DEV) + 0.5).to(F16)
    tables = kvc.profile(cd, prof)
    enc = kvc.encode(cd, tables, kv, [0, 1, 0])
    n_q, steps = 21, 3
    total = T + n_q + steps
    width = (total + page - 1) // page
    n_pages = 2 * width + 5
    pd = kvc.make_paged_desc(L, heads, hk, d, page, n_pages, F16, BF16)
    pool = torch.full(pd.pool_shape, float("nan"), dtype=F16, device=DEV)
    first = 3  # sequence 0: pages 3, 4, ...; sequence 1: the others, shuffled
    rest = [i for i in range(n_pages) if not first <= i < first + width]
    perm = torch.randperm(len(rest), generator=g, device=DEV).tolist()
    table = torch.tensor([list(range(first, first + width)), [rest[i] for i in perm][:width]],
                         dtype=torch.int32, device=DEV)
    refs = kvc.chunk_refs(enc, first_tokens=[first * page + 1500 * k for k in range(3)])
    kvc.decode(cd, tables, refs, pool.shape[2], out=pool)
    flat = kvc.decode(cd, tables, kvc.chunk_refs(enc), T)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvc.page_in_async(pd, flat, 0, pool, table[1], 0, T, status)
    kvc.read_status(status, "page_in")

    rope = kvc.Rope(kvc.rope_table(total, d, device=DEV))
    lens = torch.tensor([T, T], dtype=torch.int32, device=DEV)
    q_start = torch.tensor([0, n_q, 2 * n_q], dtype=torch.int32, device=DEV)
    prompt = kvc.PagedBatch(table, lens, q_start=q_start, max_len=total)
    single = kvc.PagedBatch(table, lens, max_len=total)
    wp, ws = kvc.PagedWorkspace(pd, prompt, 2 * n_q), kvc.PagedWorkspace(pd, single)
    done = T
    for n, batch, wsp, attend in [(n_q, prompt, wp, kvc.attend_prompt_async)] + [
            (1, single, ws, kvc.attend_async)] * steps:
        one = torch.randn((n, heads + 2 * hk, d), generator=g, device=DEV).to(BF16)
        rows = torch.cat([one, one])  # both sequences get the same tokens
        done += n
        lens.fill_(done)
        for layer in range(L):
            q = torch.empty_like(rows[:, :heads].contiguous())
            out, lse = torch.empty_like(q), torch.empty((2 * n, heads), device=DEV)
            kvc.append_async(pd, batch, layer, pool, rows[:, heads:heads + hk],
                             rows[:, heads + hk:], wsp, rope=rope, q=rows[:, :heads], q_out=q)
            attend(pd, batch, layer, pool, q, out, wsp, lse=lse)
            kvc.read_status(wsp.status, "step")
            # each copy by itself: the same bits wherever its pages lie
            alone = []
            for b in range(2):
                qs = None if n == 1 else torch.tensor([0, n], dtype=torch.int32, device=DEV)
                one_batch = kvc.PagedBatch(table[b:b + 1], lens[b:b + 1], q_start=qs,
                                           max_len=total)
                one_ws = kvc.PagedWorkspace(pd, one_batch, n)
                o1, e1 = torch.empty_like(out[:n]), torch.empty_like(lse[:n])
                attend(pd, one_batch, layer, pool, q[b * n:(b + 1) * n], o1, one_ws, lse=e1)
                kvc.read_status(one_ws.status, "alone")
                alone.append((o1, e1))
            assert torch.equal(alone[0][0], alone[1][0])
            assert torch.equal(alone[0][1], alone[1][1])
            s = ref.slots(table[1], done, page, DEV)
            k = pool[layer, 0, s].view(-1, hk, d)
            v = pool[layer, 1, s].view(-1, hk, d)
            assert torch.equal(pool[layer, 0, s[:T]], flat[layer, 0].view(F16))
            o, e, bo, be = ref.attend(q[:n], k, v, list(range(done - n, done)), d ** -0.5, 0, F16,
                                      BF16)
            for got, got_e in ((out[:n], lse[:n]), (out[n:], lse[n:]), alone[0]):
                assert bool(((got.double() - o).abs() <= bo).all())
                assert bool(((got_e.double() - e).abs() <= be).all())
    # evicted again: both copies give the same containers
    blobs = []
    for b in range(2):
        back = torch.empty((L, 2, total, c), dtype=F16, device=DEV)
        kvc.page_out_async(pd, pool, table[b], 0, total, back, 0, status)
        kvc.read_status(status, "page_out")
        assert torch.equal(back[:, :, :T], flat.view(F16))
        blobs.append(kvc.encode(cd, tables, back, [1, 1, 0]).blob)
    assert torch.equal(blobs[0], blobs[1])
