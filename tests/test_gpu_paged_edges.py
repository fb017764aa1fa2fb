"""The paged-cache operators on the GPU where a plan, a value or a size is
unusual."""
import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import paged_ref as ref
from test_gpu_paged import BF16, DEV, F16, Setup, _attend, _check_attend, _gen

pytestmark = pytest.mark.gpu


# heads, kv_heads, head_dim: one head a workgroup (four waves to it), two, four
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(4, 1, 64), (6, 2, 128), (8, 8, 256)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens", [[90, 33, 500, 1], [1410, 33, 700, 65]])  # whole sequences; cut
@pytest.mark.parametrize("window", [0, 24, 600])
def test_single_tokens_and_nonfinite_values(heads, kv_heads, head_dim, dtype, lens, window):
    """Keys and values before the window have no effect, whatever they hold;
    an infinity in the last visible value, in a tile that it does not fill,
    gives an infinity in its dimensions and nothing in the others."""
    st = Setup(lens, [1] * len(lens), heads, kv_heads, head_dim, 16, dtype, dtype, single=True)
    last = []
    for b, m in enumerate(lens):
        s = st.slots(b)
        if window and m > window:
            hidden = s[:m - window]
            st.pool[1, :, hidden[::2]] = float("nan")
            st.pool[1, 1, hidden[1::2]] = float("inf")
        last.append(int(s[m - 1]))
    out, lse = _attend(st, window)
    out_inf, lse_inf = _attend_with_last(st, last, window)
    odd = torch.zeros(head_dim, dtype=torch.bool, device=DEV)
    odd[1::3] = True
    for b, m in enumerate(lens):
        k, v = st.cached(b)
        o, e, bo, be = ref.attend(st.q[b:b + 1], k, v, [m - 1], head_dim ** -0.5, window, dtype,
                                  dtype)
        assert bool(((out[b].double() - o[0]).abs() <= bo[0]).all()), (b, m)
        assert bool(((lse[b].double() - e[0]).abs() <= be[0]).all()), (b, m)
        assert bool((out_inf[b][:, odd] == float("inf")).all()), (b, m)
        assert torch.equal(out_inf[b][:, ~odd], out[b][:, ~odd])
        assert torch.equal(lse_inf[b], lse[b])


def _attend_with_last(st, last, window):
    """The same call with +infinity in dimensions 1, 4, 7, ... of the sequences'
    last values (taken back afterwards)."""
    d = st.head_dim
    rows = st.pool[1, 1].view(-1, st.kv_heads, d)
    kept = rows[last].clone()
    bad = kept.clone()
    bad[..., 1::3] = float("inf")
    rows[last] = bad
    got = _attend(st, window)
    rows[last] = kept
    return got


@pytest.mark.parametrize("heads,kv_heads,n_seqs,long", [
    (4, 1, 96, 3000),    # steps of 64 tokens, four waves to a head
    (64, 64, 64, 5000),  # steps of 1,024 tokens, four heads to a workgroup
])
def test_plans_for_lengths_to_2_30(heads, kv_heads, n_seqs, long):
    """max_len left out over a table that could hold 2^30 tokens a sequence:
    steps of more than 32 tokens, so that a call's number them in 31 bits.
    The sequences share a few pages; entries past a length are never read."""
    d, page, n_pages = 64, 2048, 6
    desc = kvc.make_paged_desc(1, heads, kv_heads, d, page, n_pages, F16, F16)
    g = _gen(3)
    pool = torch.randn(desc.pool_shape, generator=g, device=DEV).to(F16)
    lens = [(37 * i) % 90 + 1 for i in range(n_seqs)]
    lens[5], lens[n_seqs // 2], lens[-1], lens[7] = long, long // 2 + 3, 1100, 0
    table = torch.full((n_seqs, 2 ** 30 // page), -(2 ** 31), dtype=torch.int32, device=DEV)
    for b, m in enumerate(lens):
        need = (m + page - 1) // page
        table[b, :need] = torch.randint(0, n_pages, (need,), generator=g, device=DEV,
                                        dtype=torch.int32)
    lens_dev = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn((n_seqs, heads, d), generator=g, device=DEV).to(F16)
    got = []
    for max_len in (None, max(lens)):
        batch = kvc.PagedBatch(table, lens_dev, max_len=max_len)
        wsp = kvc.PagedWorkspace(desc, batch)
        out = torch.full_like(q, 7.0)
        lse = torch.full((n_seqs, heads), 7.0, device=DEV)
        kvc.attend_async(desc, batch, 0, pool, q, out, wsp, lse=lse)
        kvc.read_status(wsp.status, "attend")
        got.append((out, lse))
    for b, m in enumerate(lens):
        if m == 0:
            for out, lse in got:
                assert bool((out[b] == 0).all()) and bool((lse[b] == float("-inf")).all())
            continue
        s = ref.slots(table[b], m, page, DEV)
        k, v = (pool[0, kv, s].view(m, kv_heads, d) for kv in range(2))
        o, e, bo, be = ref.attend(q[b:b + 1], k, v, [m - 1], d ** -0.5, 0, F16, F16)
        for out, lse in got:
            assert bool(((out[b].double() - o[0]).abs() <= bo[0]).all()), (b, m)
            assert bool(((lse[b].double() - e[0]).abs() <= be[0]).all()), (b, m)


@pytest.mark.parametrize("window", [0, 1, 64, 300])
@pytest.mark.parametrize("heads,kv_heads,lens,new", [
    (8, 1, [700, 4, 90], [4, 4, 3]),       # 128-row tiles
    (128, 1, [70, 9, 800], [9, 9, 9]),     # 256-row tiles
    (40, 1, [600, 3, 1500], [1, 1, 1]),    # single tokens of more than 16 heads
    (8, 2, [600, 3, 1500], [1, 1, 1]),     # single tokens, 16-row tiles
])
def test_bound_of_the_lengths_far_above_them(heads, kv_heads, lens, new, window):
    """max_len 131,072: most splits of a tile see no token."""
    single = max(new) == 1
    st = Setup(lens, new, heads, kv_heads, 64, 16, F16, F16, single=single)
    wide = torch.full((len(lens), 131072 // 16), -1, dtype=torch.int32, device=DEV)
    wide[:, :st.table.shape[1]] = st.table
    st.batch = kvc.PagedBatch(wide, st.lens, q_start=st.batch.q_start)
    st.wsp = kvc.PagedWorkspace(st.desc, st.batch, st.n_tok)
    st.wsp.ws.fill_(0xFF)
    out, lse = _attend(st, window, prompt=not single)
    _check_attend(st, out, lse, window)


@pytest.mark.parametrize("heads,new", [(2, 40), (128, 9)])  # 128 and 256 rows a workgroup
def test_prompt_long_tail_of_small_probabilities(heads, new):
    """One token far above thousands of others whose weights are small binary16
    numbers of the largest, or far below its smallest step, yet sum to a part
    of the output that its bound does not cover."""
    m, d = 4097, 64
    st = Setup([m], [new], heads, 1, d, 16, F16, F16)
    s = st.slots(0)
    st.pool[1, 0, s] = 0.0
    st.pool[1, 0, s[100], 0] = 1.0
    st.pool[1, 1, s] = 1.0
    st.pool[1, 1, s[100]] = 0.0
    k, v = st.cached(0)
    scale = 1.3
    for q0 in (8.0, 16.0):  # exp(-10.4) = 2^-15, exp(-20.8) = 2^-30
        st.q.zero_()
        st.q[:, :, 0] = q0
        out, lse = _attend(st, scale=scale, prompt=True)
        o, e, bo, be = ref.attend(st.q[:, :1], k, v, list(range(m - new, m)), scale, 0, F16, F16,
                                  shift=11)
        assert bool(((out.double() - o).abs() <= bo).all())
        assert bool(((lse.double() - e).abs() <= be).all())
        assert bool((out > 0).all()) and bool((bo < o).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,new", [(4, 1), (40, 1), (4, 50), (128, 20)])
def test_scales_at_the_ends_of_binary32(heads, new, dtype):
    """A subnormal scale makes all scores (nearly) equal and hides hidden
    tokens still; the largest scale gives finite scores on small products."""
    st = Setup([700], [new], heads, 1, 64, 16, dtype, dtype, single=new == 1)
    out, lse = _attend(st, 33, scale=1e-40, prompt=new > 1)
    _check_attend(st, out, lse, 33, scale=1e-40)
    k, v = st.cached(0)
    tiny = 2.0 ** -14
    st.pool[1, 0, st.slots(0)] = tiny
    st.q.fill_(tiny)
    for scale in (2.358e38, -2.358e38):
        out, lse = _attend(st, scale=scale, prompt=new > 1)
        for i in range(new):
            n = 700 - new + 1 + i
            # equal scores: weights of 1 / n, exact powers of two before the
            # quotient; binary32 sums of n terms and one rounding
            mean, mag = v[:n, 0].double().mean(0), v[:n, 0].double().abs().mean(0)
            bound = (2 * n + 8) * ref.F32 * mag + ref.half_step(dtype) * (mean.abs() + mag * 2e-4)
            assert bool(((out[i].double() - mean).abs() <= bound + 2.0 ** -25).all()), i
        # 64 equal products, exact; the scale rounded and multiplied
        want = 64 * tiny * tiny * scale
        assert bool(((lse.double() - want).abs() <= 8 * ref.F32 * abs(want)).all())


@pytest.mark.parametrize("n_seqs", [64, 70])  # one and two search steps
def test_q_start_that_overlaps_itself_in_256_row_tiles(n_seqs):
    """Every other sequence claims all rows (1,280 and more a sequence on
    average): reported, and the call ends."""
    heads, new = 128, 10
    st = Setup([40] * n_seqs, [new] * n_seqs, heads, 1, 64, 16, F16, F16)
    n = n_seqs * new
    assert n * heads // n_seqs >= 1024
    st.batch.q_start[0::2] = 0
    st.batch.q_start[1::2] = n
    out = torch.zeros((n, heads, 64), dtype=F16, device=DEV)
    kvc.attend_prompt_async(st.desc, st.batch, 1, st.pool, st.q, out, st.wsp)
    assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
