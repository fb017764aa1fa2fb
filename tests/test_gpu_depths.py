"""Positions of a drafted tree's tokens that are negative, with and without a
rotation that would use them."""
import pytest
import torch

import kv_cache_compression_decode_amd as kvc
from test_gpu_drafts import BF16, DEV, F16, Drafts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("io,cache", [(F16, F16), (BF16, F16), (BF16, BF16)])
def test_negative_position(rotary, normed, io, cache):
    """The token is left out, keys, values and query, and the error stored; the
    others are written."""
    st = Drafts([40, 20], [9, 5], 4, 2, 64, 16, io, cache)
    norm = kvc.HeadNorm(*[torch.ones(64, device=DEV)] * 2) if normed else None
    rope = kvc.Rope(kvc.rope_table(64, rotary)) if rotary else None
    before = st.pool.clone()
    for value in (-32, -100, -2 ** 31):  # the sequence's first new position is 31
        st.tree.depth[3] = value
        st.pool.copy_(before)
        q_out = torch.full_like(st.q, 7.0)
        kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, norm=norm, rope=rope,
                         tree=st.tree, q=st.q, q_out=q_out)
        assert int(st.wsp.status.item()) == kvc.ERR_SHAPE
        st.wsp.status.zero_()
        s = st.slots(0)
        assert torch.equal(st.pool[1, :, s[34]], before[1, :, s[34]])
        assert bool((q_out[3] == 7.0).all())
        for i in (0, 2, 4, 8):
            assert torch.equal(st.pool[1, 1, s[31 + i]], st.v[i].flatten().to(cache))
            assert not bool((q_out[i] == 7.0).all())
    # position 0 is the least that is allowed
    st.tree.depth[3] = -31
    kvc.append_async(st.desc, st.batch, 1, st.pool, st.k, st.v, st.wsp, norm=norm, rope=rope,
                     tree=st.tree)
    kvc.read_status(st.wsp.status, "append")
    assert torch.equal(st.pool[1, 1, st.slots(0)[34]], st.v[3].flatten().to(cache))
