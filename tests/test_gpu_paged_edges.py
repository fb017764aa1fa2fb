"""The paged-cache operators on the GPU where a plan, a value or a size is
unusual."""
import pytest
import torch

import paged_ref as ref
from test_gpu_paged import F16, Setup, _attend

pytestmark = pytest.mark.gpu


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
