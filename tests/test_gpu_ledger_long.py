"""The page ledger with rows of many pages: more than a wave, more than a
workgroup takes at a time."""
import pytest

import kv_cache_compression_decode_amd as kvc
from test_gpu_ledger import State, _i32

pytestmark = pytest.mark.gpu


def test_fork_between_long_and_short_rows():
    """Rows of 3 to 700 pages take each other's places, the longer one as the
    source and as the destination; what a row gave up is then handed out."""
    st = State(8, 700, 1, 5000)
    st.resize([700, 65, 300, 3, 0, 257, 129, 64])
    st.check()
    for src, dst in (([0], [1]), ([3], [2]), ([5, 5], [4, 3]), ([6, 0], [5, 7]), ([7], [0]),
                     ([1, 2, 2], [6, 0, 4]), ([1, 1, 1], [2, 3, 5])):
        st.fork(src, dst)
        st.check()
    st.resize([350, 700, 699, 256, 600, 700, 0, 64])
    st.check()
    st.resize([0] * 8)
    st.check()
    assert not bool(st.ledger.refs.any())


def test_many_forks_of_long_rows():
    """All forks of a call at once, half of them from short to long rows and
    half from long to short ones."""
    rows, entries = 128, 330
    st = State(rows, entries, 2, 32000)
    lens = [(1 + (r * 83) % 330) * 2 for r in range(rows)]
    for step in range(4):
        st.resize(lens)
        st.check()
        order = sorted(range(rows), key=lambda r: lens[r])
        low, high = order[:rows // 2], order[rows // 2:]
        a, b = low[:32], high[:32]  # as sources
        st.fork(a + b, high[32:] + low[32:])
        st.check()
        lens = [(1 + (r * 83 + step * 57) % 330) * 2 - r % 2 for r in range(rows)]


@pytest.mark.parametrize("rows,entries,page", [(4, 1200, 1), (7, 900, 4), (300, 40, 3)])
def test_thousands_of_pages_in_a_call(rows, entries, page):
    """Rows grow from nothing to all that the table holds in one call, are
    forked, shrink, and grow again."""
    top = entries * page
    st = State(rows, entries, page, rows * entries + 10)
    st.resize([top - r % page for r in range(rows)])
    assert sum(x > 0 for x in st.plain.refs) > 2048
    st.check()
    half = rows // 2
    st.fork(list(range(half)), list(range(half, 2 * half)))
    st.check()
    st.resize([(r * 77) % (top // 2) for r in range(rows)])
    st.check()
    st.fork([0], [rows - 1])
    st.resize([top - (3 * r) % (2 * page) for r in range(rows)])
    st.check()
    st.resize([0] * rows)
    st.check()
    assert not bool(st.ledger.refs.any())


def test_copies_behind_thousands_of_pages():
    """Rows that copy a shared page after others have taken more than 2,048
    pages, and rows that take theirs after those."""
    st = State(8, 1300, 3, 9000)
    st.resize([0, 0, 0, 100, 0, 0, 50, 0])
    st.fork([3, 3, 6], [4, 5, 7])
    st.check()
    st.resize([3900, 3899, 0, 101, 3898, 100, 52, 51])
    st.check()
    # row 5 still holds the page at its old length, so rows 3 and 4 have copies
    assert len(st.plain.copies) == 3 and st.plain.copies[0][1] > 2048
    st.resize([1, 2, 3900, 3, 3900, 3900, 0, 3900])
    st.check()


def test_few_free_pages_among_many():
    """A pool of 50,000 pages of which others hold all but some, the last ones
    among them: they are found, and one too many is refused."""
    st = State(3, 100, 2, 50000)
    free = [7, 16383, 16384, 16385, 32768, 40000, 49151, 49152, 49998, 49999]
    st.plain.refs = [0 if i in free else 1 for i in range(50000)]
    st.ledger.refs.copy_(_i32(st.plain.refs))
    st.resize([7, 0, 3])
    st.check()
    kvc.resize_async(st.ledger, st.pool, _i32([7, 9, 3]))  # 5 of 4
    assert int(st.ledger.status.item()) == kvc.ERR_CAPACITY
    st.ledger.status.zero_()
    st.check()
    st.resize([8, 8, 4])
    st.check()
    assert 0 not in st.plain.refs
    st.resize([0, 3, 4])
    st.fork([1], [0])
    st.resize([4, 5, 4])  # a copy and a page
    st.check()
