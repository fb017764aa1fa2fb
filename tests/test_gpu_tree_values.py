"""Keys that are not finite in the context of a drafted tree, wherever the
context is cut: what every token of the tree sees shows in every one of them."""
import pytest
import torch

from test_gpu_drafts import BF16, F16, Drafts

pytestmark = pytest.mark.gpu

# Each is a shape whose long sequence is cut among several workgroups or waves:
# 16 and 32 rows to a KV head, 128-row and 256-row tiles, few and many parts.
CUT = [
    # heads, kv_heads, head_dim, io, cache, lens, new
    (1, 1, 64, F16, F16, [1025], [1]),
    (2, 2, 128, BF16, F16, [1300], [9]),
    (8, 8, 128, BF16, BF16, [4100, 700, 30], [16, 3, 5]),
    (16, 4, 128, F16, F16, [3000, 900], [8, 7]),
    (8, 2, 96, F16, F16, [2100, 90], [20, 11]),
    (64, 8, 128, F16, F16, [5026], [26]),
    (64, 8, 64, BF16, BF16, [4000, 1500], [60, 17]),
    (2, 2, 256, F16, F16, [1200], [12]),
    (6, 2, 256, BF16, F16, [1500, 300], [30, 8]),
]


@pytest.mark.parametrize("heads,kv_heads,head_dim,io,cache,lens,new", CUT)
def test_nan_keys_of_the_context(heads, kv_heads, head_dim, io, cache, lens, new):
    """Runs of NaN keys in one KV head, some of them a cut's whole share: that
    head's rows and log-sum-exps of the sequence are NaN, all others as before."""
    st = Drafts(lens, new, heads, kv_heads, head_dim, 16, io, cache)
    whole, whole_lse = st.attend()
    keys = st.pool[1, 0].view(-1, kv_heads, head_dim)
    s, base, g = st.slots(0), lens[0] - new[0], heads // kv_heads
    head = kv_heads - 1
    kept = keys.clone()
    for first, n in ((0, 96), (0, 128), (0, 256), (0, 512), (128, 128), (96, 96), (256, 256),
                     (base - 32, 32), (base - 130, 128), (0, base), (base // 2, 1)):
        keys[s[first:first + n], head] = float("nan")
        out, lse = st.attend()
        keys.copy_(kept)
        mine = slice(head * g, (head + 1) * g)
        assert bool(out[: new[0], mine].isnan().all()), (first, n)
        assert bool(lse[: new[0], mine].isnan().all()), (first, n)
        for got, want in ((out, whole), (lse, whole_lse)):
            got[: new[0], mine] = want[: new[0], mine]
            assert torch.equal(got, want), (first, n)


@pytest.mark.parametrize("heads,kv_heads,head_dim,io,cache,lens,new", CUT)
def test_scores_of_minus_infinity(heads, kv_heads, head_dim, io, cache, lens, new):
    """Context tokens whose score is minus infinity in every row have no weight:
    the outputs are those of the tree with other values and keys in their place
    that are as light.  All of them: the rows' own tokens alone."""
    st = Drafts(lens, new, heads, kv_heads, head_dim, 16, io, cache)
    st.q[:, :, 0] = st.q[:, :, 0].abs() + 0.5
    keys = st.pool[1, 0].view(-1, kv_heads, head_dim)
    s, base = st.slots(0), lens[0] - new[0]
    kept = keys.clone()
    for first, n in ((0, 96), (0, 128), (0, 256), (128, 128), (base - 32, 32), (0, base)):
        results = []
        for light in (float("-inf"), -60000.0):  # scores below -3,000: exp2 of them is 0
            keys[s[first:first + n], :, 0] = light
            results.append(st.attend())
            keys.copy_(kept)
        for a, b in zip(*results):
            assert torch.equal(a, b), (first, n)
        assert bool(results[0][0][: new[0]].isfinite().all())
