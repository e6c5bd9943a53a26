"""The block operators where they can go wrong, on the GPU against the float64 oracle (oracle/block.py). Tolerances as in
test_gpu_block.py, or exact, unless a test derives its own."""
import numpy as np
import pytest

from oracle import block as ob
from tests.test_gpu_block import E, SUB, U, Setup, bk, check_attention, close, dev  # noqa: F401  (bk: the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ small weights
SINKS = [  # new tokens, length, query heads, kv heads, dim, token of the large key
    ([1], [3000], 4, 1, 128, 5),
    ([1], [700], 2, 2, 64, 699),
    ([16], [3000], 4, 1, 128, 0),
    ([100], [3000], 4, 1, 128, 5),                      # many rows, split over the cache
    ([300], [2500], 4, 1, 64, 70),
    ([513], [2600], 8, 4, 128, 3),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,lens,hq,hk,D,sink", SINKS)
def test_attention_keeps_small_weights(bk, new, lens, hq, hk, D, sink, fmt):
    """One key takes nearly all the weight and its value is zero: what is left is the sum of thousands of weights of
    2^-24.5 each, which together are the output.

    Weights are rounded to fp16 relative to a reference at most 2^11 below the largest, so 2^-24.5 of it is a normal fp16
    number: the tolerance has no part that grows with the length. The scores' error is d as in test_gpu_block.py."""
    print("sink", new, lens, hq, hk, D, sink, fmt, flush=True)
    st = Setup(bk, lens, hk, D, fmt, seed=sum(lens) + D + sink)
    gap = 24.5 * np.log(2)                              # in units of the scaled scores

    def values(s, k, v):
        k[:] = 0
        k[sink] = np.float16(gap / D ** 0.5)            # the query is all ones, the scale D^-1/2
        v[:] = (100 + 10 * st.g.standard_normal(v.shape)).astype(np.float16)
        v[sink] = 0
    st.fill(values)
    T = sum(new)
    q = dev(np.ones((T, hq, D), np.float16))
    got = bk.mq_kv_attention(q, st.cache, st.batch(new)).cpu().numpy()
    L, n = lens[0], new[0]
    for i in sorted({0, n // 2, n - 1}):
        for h in range(hq):
            k, v = st.ref.read(L, st.tables[0], st.slots[0], h * hk // hq)
            vis = L - n + i + 1
            o, pv, sa = ob.attend(np.ones(D), k, v, vis, D ** -0.5)
            assert vis > sink and np.all(o > 64 * SUB)
            d = (D + 8) * E * sa
            close(got[i, h], o, U * np.abs(o) + SUB + (U + 2 * d + (D + 8 + L / 16) * E) * pv, f"token {i} head {h}")
