"""Attention with a sliding window and sinks on the GPU against 64-bit forms:
single tokens and prompts, gaps and edges at every place of a tile, and values
that are not finite in hidden tokens."""
import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import serve_ref
from test_gpu_paged import BF16, DEV, F16, Setup

pytestmark = pytest.mark.gpu


def _attend(st, window, sinks, single):
    out = torch.full((st.n_tok, st.heads, st.head_dim), 7.0, dtype=st.io, device=DEV)
    lse = torch.full((st.n_tok, st.heads), 7.0, device=DEV)
    f = kvc.attend_async if single else kvc.attend_prompt_async
    f(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, window=window, lse=lse, sinks=sinks)
    kvc.read_status(st.wsp.status, "attend")
    return out, lse


def _check(st, out, lse, window, sinks, shift, skip=()):
    """Rows (sequence, new token) in skip are not compared."""
    for b, (m, n) in enumerate(zip(st.lens_host, st.new_host)):
        a = st.start[b]
        k, v = st.cached(b)
        seen = serve_ref.sinks_seen(list(range(m - n, m)), m, window, sinks, DEV)
        o, e, bo, be = serve_ref.attend_seen(st.q[a:a + n], k, v, seen, st.head_dim ** -0.5,
                                             st.cache, st.io, shift)
        for i in range(n):
            if (b, i) in skip:
                continue
            got, got_e = out[a + i].double(), lse[a + i].double()
            if not bool(seen[i].any()):
                assert bool((got == 0).all()) and bool((got_e == float("-inf")).all())
                continue
            assert bool(((got - o[i]).abs() <= bo[i]).all()), (b, i, m, n)
            assert bool(((got_e - e[i]).abs() <= be[i]).all()), (b, i, m, n)
    a = st.start[-1]
    assert bool((out[a:] == 7.0).all()) and bool((lse[a:] == 7.0).all())


def _hide(st, window, sinks):
    """NaN and infinities where no row sees: between the sinks and the window
    of each sequence's first new token."""
    for b, (m, n) in enumerate(zip(st.lens_host, st.new_host)):
        lo = max(m - n + 1 - window, 0) if window else 0
        if lo > sinks:
            s = st.slots(b)[sinks:lo]
            st.pool[1, :, s] = float("nan")
            st.pool[1, 1, s[::2]] = float("inf")


SINGLE = [
    # heads, kv_heads, head_dim, page, io, cache, lens, window, sinks
    (8, 2, 64, 16, F16, F16, [1, 2, 33, 34, 100, 129, 700], 32, 4),
    (64, 8, 128, 16, F16, F16, [5000], 1024, 4),
    (64, 8, 128, 20, BF16, F16, [3001, 0, 1, 65, 900], 257, 33),
    (4, 4, 128, 7, BF16, BF16, [513, 90, 91, 92], 1, 1),
    (6, 2, 256, 48, BF16, F16, [700, 3, 64, 1300], 500, 300),
    (14, 2, 96, 1, F16, F16, [100, 257, 40], 33, 64),
    # sinks that reach the window, and pass the whole sequence
    (5, 5, 64, 10, F16, F16, [600, 90, 1100], 64, 536),
    (5, 5, 64, 10, F16, F16, [600, 90, 1100], 64, 4000),
    # more than 16 heads to a KV head: tiles of 128 rows, and short ones
    (40, 2, 128, 16, F16, F16, [3000, 1, 800], 300, 5),
    (20, 1, 96, 16, BF16, BF16, [400, 33, 0], 100, 17),
    # more sequences than a search step takes
    (4, 1, 64, 16, F16, F16, [(i * 37) % 23 * 30 + i % 5 for i in range(300)], 200, 3),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,window,sinks", SINGLE)
def test_sinks_single(heads, kv_heads, head_dim, page, io, cache, lens, window, sinks):
    st = Setup(lens, [1] * len(lens), heads, kv_heads, head_dim, page, io, cache, single=True)
    _hide(st, window, sinks)
    out, lse = _attend(st, window, sinks, True)
    # binary16 probabilities are scaled by 2^11 in the larger tiles
    _check(st, out, lse, window, sinks, 11 if heads // kv_heads > 16 else 14)


PROMPT = [
    # heads, kv_heads, head_dim, page, io, cache, lens, new, window, sinks
    (8, 2, 64, 16, F16, F16, [5, 40, 133], [5, 3, 133], 20, 4),
    (4, 4, 128, 16, BF16, BF16, [130, 1, 700], [130, 1, 129], 100, 1),
    (16, 2, 128, 20, BF16, F16, [900, 0, 65], [70, 2, 65], 64, 70),
    (6, 2, 256, 7, F16, F16, [400, 90], [50, 33], 33, 40),
    (5, 5, 96, 16, F16, F16, [600, 300], [300, 300], 31, 64),
    (8, 8, 64, 64, BF16, F16, [1500], [4], 200, 16),
    # 256-row tiles
    (64, 8, 128, 16, F16, F16, [700, 260], [140, 150], 128, 3),
    (8, 1, 64, 10, BF16, BF16, [300], [300], 1, 2),
    # padding rows before the first token
    (4, 2, 64, 16, F16, F16, [3, 2], [5, 2], 2, 1),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,io,cache,lens,new,window,sinks", PROMPT)
def test_sinks_prompt(heads, kv_heads, head_dim, page, io, cache, lens, new, window, sinks):
    st = Setup(lens, new, heads, kv_heads, head_dim, page, io, cache, spare=2)
    _hide(st, window, sinks)
    out, lse = _attend(st, window, sinks, False)
    _check(st, out, lse, window, sinks, 11)


def test_sinks_prompt_infinite_value_seen_by_some():
    """A value that is not finite reaches the rows that see it and no other:
    a sink in the same tile, a token that has left some rows' windows."""
    st = Setup([300], [120], 8, 2, 64, 16, F16, F16)
    window, sinks = 50, 10
    s = st.slots(0)
    st.pool[1, 1, s[200]] = float("inf")  # in the windows of rows 200 .. 249
    out, lse = _attend(st, window, sinks, False)
    hit = {(0, i) for i in range(120) if 200 <= 180 + i < 250}
    _check(st, out, lse, window, sinks, 11, skip=hit)
    for _, i in hit:
        assert not bool(torch.isfinite(out[i].double()).any())


@pytest.mark.parametrize("single", [True, False])
def test_without_sinks_or_window_nothing_changes(single):
    new = [1, 1, 1] if single else [3, 200, 9]
    st = Setup([900, 1300, 9], new, 16, 4, 128, 16, F16, F16, single=single)
    f = kvc.attend_async if single else kvc.attend_prompt_async
    for window, sinks in ((0, 5), (100, 0)):
        want = torch.zeros((st.n_tok, 16, 128), dtype=F16, device=DEV)
        got = torch.zeros_like(want)
        f(st.desc, st.batch, 1, st.pool, st.q, want, st.wsp, window=window)
        f(st.desc, st.batch, 1, st.pool, st.q, got, st.wsp, window=window, sinks=sinks)
        kvc.read_status(st.wsp.status, "attend")
        assert torch.equal(got, want)


def test_sinks_bad_page_and_length():
    for damage in ("page", "length"):
        st = Setup([900, 300], [1, 1], 8, 2, 64, 16, F16, F16, single=True)
        if damage == "page":
            st.table[0, 0] = st.n_pages  # a sink's page
        else:
            st.lens[1] = 901
        out = torch.zeros((2, 8, 64), dtype=F16, device=DEV)
        kvc.attend_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, window=64, sinks=4)
        with pytest.raises(kvc.KvcError) as e:
            kvc.read_status(st.wsp.status, "attend")
        assert e.value.code == kvc.ERR_SHAPE


@pytest.mark.parametrize("single", [True, False])
def test_sinks_captured_and_replayed_as_lengths_grow(single):
    new = [1, 1] if single else [4, 130]
    st = Setup([900, 700], new, 8, 2, 64, 16, F16, F16, single=single)
    out = torch.zeros((st.n_tok, 8, 64), dtype=F16, device=DEV)
    want = torch.zeros_like(out)
    f = kvc.attend_async if single else kvc.attend_prompt_async
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        f(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, window=90, sinks=7)
        with torch.cuda.graph(graph, stream=side):
            f(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp, window=90, sinks=7)
    torch.cuda.current_stream().wait_stream(side)
    wsp = kvc.PagedWorkspace(st.desc, st.batch, st.n_tok)
    for lens in ([900, 700], [500, 131], [131, 699], [140, 140]):
        st.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.zero_()
        graph.replay()
        f(st.desc, st.batch, 1, st.pool, st.q, want, wsp, window=90, sinks=7)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and bool((out != 0).any())
    kvc.read_status(st.wsp.status, "attend")
