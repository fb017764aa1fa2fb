"""CPU checks: what fork and resize read may not lie in the ledger that they
write (refused before anything is launched)."""
import pytest

import kv_cache_compression_decode_amd as kvc
from test_more_host import L, _desc, _fork, _ledger, _resize  # noqa: F401 (L is a fixture)
from test_paged_host import A

# 5 rows of 10 entries, 100 pages
PLACES = [("table", 2 * A, 50), ("lens", 3 * A, 5), ("refs", 4 * A, 100)]
APART = {name: at for name, at, _ in PLACES}


@pytest.mark.parametrize("name,at,n", PLACES)
def test_overlaps(L, name, at, n):  # noqa: F811
    g = _ledger(**APART)
    # three entries of src or dst, five of new_lens: the first and the last place
    # that share one with the array
    for first in (at - 4 * 2, at, at + 4 * (n - 1)):
        assert _fork(L, g=g, src=first, dst=A) == kvc.ERR_SHAPE
        assert _fork(L, g=g, src=A, dst=first) == kvc.ERR_SHAPE
    for first in (at - 4 * 4, at, at + 4 * (n - 1)):
        assert _resize(L, g=g, lens=first) == kvc.ERR_SHAPE


def test_empty_ledger(L):  # noqa: F811
    assert _fork(L, g=_ledger(rows=0), n=0) == 0 and _resize(L, g=_ledger(rows=0)) == 0
