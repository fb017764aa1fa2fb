"""The paged-cache operators on the GPU where a plan, a value or a size is
unusual."""
import pytest
import torch

import kv_cache_compression_decode_amd as kvc
import paged_ref as ref
from test_gpu_paged import BF16, DEV, F16, Setup, _attend

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
