"""Trees of more than three words of mask, up to the largest that is allowed."""
import random

import pytest
import torch

import serve_ref
from test_gpu_drafts import BF16, F16, Drafts

pytestmark = pytest.mark.gpu


def _rows(n, seed):
    """Tokens at the words' edges, the last ones and some others."""
    r = random.Random(seed)
    edges = [0, 1, 62, 63, 64, 65, 127, 128, 191, 192, 255, 256, 257, n - 2, n - 1]
    return sorted({i for i in edges + [r.randrange(n) for _ in range(25)] if 0 <= i < n})


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("heads,kv_heads,head_dim,io,cache,context,new,most", [
    (2, 2, 64, F16, F16, [77, 300], [300, 20], None),
    (8, 2, 128, BF16, F16, [513, 1, 0], [700, 193, 256], None),
    (2, 1, 96, BF16, BF16, [40], [2500], None),
    (1, 1, 256, F16, F16, [30, 600], [260, 515], 4096),
    (1, 1, 128, F16, F16, [100, 50], [4096, 3], None),
    (4, 4, 64, BF16, BF16, [700, 90], [5, 9], 4096),
])
def test_attend_large_tree(kind, heads, kv_heads, head_dim, io, cache, context, new, most):
    st = Drafts([c + n for c, n in zip(context, new)], new, heads, kv_heads, head_dim, 16, io,
                cache, kind=kind, max_tokens=most)
    assert st.tree.mask.shape[1] > 3
    out, lse = st.attend()
    for b, (c, n) in enumerate(zip(context, new)):
        rows = _rows(n, b)
        seen = torch.zeros((len(rows), c + n), dtype=torch.bool, device=out.device)
        seen[:, :c] = True
        for r, i in enumerate(rows):
            path, t = [], i
            while t >= 0:
                path.append(c + t)
                t = st.parents[b][t]
            seen[r, path] = True
        k, v = st.cached(b)
        at = [st.start[b] + i for i in rows]
        o, e, bo, be = serve_ref.attend_seen(st.q[at], k, v, seen, head_dim ** -0.5, cache, io, 11)
        assert bool(((out[at].double() - o).abs() <= bo).all()), b
        assert bool(((lse[at].double() - e).abs() <= be).all()), b
