"""The page ledger with rows of many pages: more than a wave, more than a
workgroup takes at a time."""
import pytest

from test_gpu_ledger import State

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
