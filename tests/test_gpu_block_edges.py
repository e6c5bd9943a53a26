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


# ---------------------------------------------------------- scores of any size
def one_hot(bk, new, D, key, query, scale, L=190):
    """Keys whose elements all equal key(token) and queries all of one value: the weight is the largest score's alone, and
    the output its value. Each row's best key has to stand alone."""
    st = Setup(bk, [L], 1, D, "int8", seed=D + sum(new))

    def values(s, k, v):
        k[:] = np.array([key(t) for t in range(L)], np.float16)[:, None, None]
    st.fill(values)
    n = new[0]
    q = dev(np.full((n, 2, D), query, np.float16))
    got = bk.mq_kv_attention(q, st.cache, st.batch(new), scale=scale).cpu().numpy().astype(np.float64)
    k, v = st.ref.read(L, st.tables[0], st.slots[0], 0)
    for i in range(n):
        score = scale * query * k[:L - n + i + 1].sum(1)
        best = int(np.argmax(score))
        # far enough from the next one that nothing else has weight, in the precision of the scores too
        assert np.sort(score)[-1] - np.sort(score)[-2] > max(200.0, 2.0 ** -20 * np.abs(score).max())
        for h in range(2):
            close(got[i, h], v[best], 2 * U * np.abs(v[best]) + SUB, f"token {i} head {h}")


@pytest.mark.parametrize("new", [[1], [40], [70]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_of_scores_past_fp32_steps(bk, new, D, sign):
    """Scores so large that a step of fp32 is many units: the weights still come from differences of scores."""
    first, second = (52000, 60000) if sign > 0 else (1200, 300)

    def key(t):
        return {7: first, 100: second}.get(t, 300 * (10 + t * 37 % 140))
    for L in (64 + new[0], 190, 606):
        one_hot(bk, new, D, key, sign * 30000.0, D ** -0.5, L=L)


@pytest.mark.parametrize("new", [[1], [40]])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_scores_far_below_zero(bk, new, D):
    """All scores below -1e30, as a large scale makes them: the largest still takes the weight."""
    one_hot(bk, new, D, lambda t: {7: -4, 100: -1}.get(t, -(10 + t * 37 % 100)), 1.0, 1e30)


# --------------------------------------------------------- queries
@pytest.mark.parametrize("new,lens,D", [([1, 1], [40, 200], 64), ([3, 1], [3000, 70], 128), ([90, 70], [100, 1500], 64),
                                        ([80, 300], [2000, 300], 128)])
def test_attention_of_queries_that_are_not_finite(bk, new, lens, D):
    """A query with an infinite element has no finite score: its output is NaN whatever the signs, also where every score
    is -Inf, and no other row's does: those stay within two roundings to fp16 and two of the weights (values of about 1) of what
    they were (a row may move its neighbours' reference, so not every bit)."""
    import torch
    st = Setup(bk, lens, 2, D, "int8", seed=D + lens[0])

    def values(s, k, v):
        k[:, :, 3] = np.abs(k[:, :, 3]) + np.float16(0.5)   # one sign: all of its products with an infinity are alike
    st.fill(values)
    q = dev(st.g.standard_normal((sum(new), 4, D)).astype(np.float16))
    good = bk.mq_kv_attention(q, st.cache, st.batch(new))
    rows = [(0, 1, -np.inf), (new[0] - 1, 2, np.inf), (sum(new) - 1, 0, -np.inf), (new[0], 3, -np.inf)]
    for t, h, x in rows:
        q[t, h, 3] = float(x)
    for scale in (D ** -0.5, -0.25):
        if scale < 0:
            good = bk.mq_kv_attention(torch.where(q.isfinite(), q, torch.ones_like(q)), st.cache, st.batch(new), scale=scale)
        got = bk.mq_kv_attention(q, st.cache, st.batch(new), scale=scale)
        bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        for t, h, _ in rows:
            bad[t, h] = True
        assert got[bad].isnan().all(), scale
        assert ((got - good)[~bad].abs().double() <= 2 * U * good[~bad].abs().double() + 4 * U).all(), scale


def test_attention_of_infinite_queries_with_nothing_to_see(bk):
    """Zeros, as for any query that sees nothing."""
    import torch
    st = Setup(bk, [0, 2], 1, 64, "int8", seed=1)
    st.fill()
    for new in ([1, 3], [40, 50]):
        q = torch.full((sum(new), 2, 64), float("-inf"), dtype=torch.float16, device="cuda")
        got = bk.mq_kv_attention(q, st.cache, st.batch(new))
        seen = new[0] + new[1] - 2
        assert not got[:seen].any() and got[seen:].isnan().all()


# ------------------------------------------------- rows of no sequence
PADS = [  # new tokens, lengths, query heads, kv heads, dim, max_len: each way of running
    ([1, 1], [60, 40], 8, 2, 64, 64),
    ([1, 1], [6000, 700], 8, 2, 128, 6000),             # split, joined by whole workgroups
    ([1, 1, 1, 1], [1500, 700, 90, 1], 64, 16, 64, 2000),  # split in few parts
    ([100], [3000], 8, 2, 128, 3000),                   # many rows, split
    ([90, 300], [90, 900], 4, 1, 64, 900),
    ([120, 60, 200], [900, 1200, 500], 64, 32, 64, 1200),  # slices
]


@pytest.mark.parametrize("new,lens,hq,hk,D,longest", PADS)
def test_attention_leaves_rows_of_no_sequence_alone(bk, new, lens, hq, hk, D, longest):
    """Rows before the first sequence's and behind the last one's, as in a step padded to a captured size: not written,
    however the work is split and whatever the workspace holds."""
    import torch
    st = Setup(bk, lens, hk, D, "int8", seed=sum(lens))
    st.fill()
    first, last = 2, 5
    T = first + sum(new) + last
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + first
    b = bk.KVBatch(dev(cu), dev(np.array(lens, np.int32)), st.table, max(new), longest, slots=st.dslots)
    q = dev(st.g.standard_normal((T, hq, D)).astype(np.float16))
    want = bk.mq_kv_attention(q[first:T - last].contiguous(), st.cache, st.batch(new))
    ws = torch.full((max(1, bk.kv_attention_workspace(st.cache, b, T, hq)),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((T, hq, D), 7.0, dtype=torch.float16, device="cuda")
    bk.mq_kv_attention(q, st.cache, b, out=out, workspace=ws)
    assert (out[:first] == 7).all() and (out[T - last:] == 7).all()
    # the padding may change how the work is split, so not every bit: two roundings to fp16, two of the weights
    got = out[first:T - last]
    assert ((got - want).abs().double() <= 2 * U * want.abs().double() + 4 * U).all()


def test_rope_of_no_tokens(bk):
    import torch
    r = bk.Rope(64, 10)
    x, pos = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    assert bk.mq_rope(x[:0], r, pos[:0]).shape == (0, 2, 64)
    out = x[:0].clone()
    assert bk.mq_rope(torch.empty((0, 2, 64), dtype=torch.float16, device="cuda"), r, pos[:0], out=out) is out
    with pytest.raises(ValueError):
        bk.mq_rope(x[:0], r, pos)


# ----------------------------------------------------------------- streams
def freed(nbytes):
    """Addresses of a block of this size that the current stream's pool has just got back."""
    import torch
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    return range(at, at + nbytes)


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream_are_not_the_current_ones_memory(bk, raw):
    """Memory that work queued on the current stream may still use is not given to a call on another stream: its outputs
    come from that stream's pool."""
    import torch
    st = Setup(bk, [300, 90], 2, 64, "int8", seed=1)
    st.fill()
    r = bk.Rope(64, 400)
    x = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    y = torch.zeros((2, 512), dtype=torch.float16, device="cuda")
    w = torch.ones(512, dtype=torch.float16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    b = st.batch([1, 1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = side.cuda_stream if raw else side
    calls = {
        "rope": (lambda: [bk.mq_rope(x, r, pos, stream=s)], x.nbytes),
        "append": (lambda: [bk.mq_kv_append(x, x[:, :2].contiguous(), x[:, 2:].contiguous(), st.cache, b, rope=r, stream=s)], x.nbytes),
        "attention": (lambda: [bk.mq_kv_attention(x, st.cache, b, stream=s)], x.nbytes),
        "norm": (lambda: list(bk.mq_norm_residual(y, y, w, stream=s)), y.nbytes),
        "table": (lambda: [bk.Rope(64, 400, stream=s).table], 400 * 32 * 8),
    }
    for name, (call, nbytes) in calls.items():
        block = freed(nbytes)
        outs = call()
        side.synchronize()
        assert all(o.data_ptr() not in block for o in outs), name


def test_attention_on_two_streams_with_work_pending(bk):
    """Two split calls, one on the current stream behind queued work, the other on a stream of its own without a wait
    between them: each has its own workspace and gives what it gives alone."""
    import torch
    st = Setup(bk, [3000, 2500], 2, 128, "int8", seed=2)
    st.fill()
    b = st.batch([1, 1])
    q1, q2 = (dev(st.g.standard_normal((2, 8, 128)).astype(np.float16)) for _ in range(2))
    assert bk.kv_attention_workspace(st.cache, b, 2, 8) > 0
    alone = [bk.mq_kv_attention(q, st.cache, b) for q in (q1, q2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(20000000)                     # some milliseconds
        o1 = bk.mq_kv_attention(q1, st.cache, b)
        o2 = bk.mq_kv_attention(q2, st.cache, b, stream=side)
        side.synchronize()
        got2 = o2.clone()
        torch.cuda.synchronize()
        assert torch.equal(o1, alone[0]) and torch.equal(got2, alone[1])


# ------------------------------------------------------------ large launches
@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_more_rows_than_a_launch_has(bk, f32):
    """2^23 + 3 rows of 256 threads are 2^31 threads and more: the launch is cut, and the rows about the cut are right."""
    import torch
    T, W, cut = (1 << 23) + 3, 9, 1 << 23
    w = torch.ones(W, dtype=torch.float16, device="cuda")
    r = torch.full((T, W), 2.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
    y = torch.full((T, W), 1.0, dtype=torch.float16, device="cuda")
    g = torch.full((T, W), 0.5, dtype=torch.float16, device="cuda")
    for t in (0, cut - 1, cut, T - 1):
        y[t] = torch.arange(W, device="cuda").half()
    r2, h = bk.mq_norm_residual(y, r, w, gate=g, eps=0.0)
    want = 2.0 + 0.5 * y.float()
    assert torch.equal(r2.float(), want)
    norm = want * (want.square().mean(1, keepdim=True)).rsqrt()
    assert ((h.float() - norm).abs() <= U * norm + 64 * E * norm).all()


# ------------------------------------- whole turns of the kernel for many rows
@pytest.mark.parametrize("new,lens,hk,D", [([130, 300], [1000, 1700], 2, 64), ([100, 200], [1300, 700], 2, 128),
                                           ([130, 300], [900, 950], 2, 128), ([120, 200], [900, 1200], 32, 64)])
def test_bad_blocks_in_the_middle_of_a_prompt(bk, new, lens, hk, D):
    """A vector that is not finite, and a block that does not exist, among whole blocks far from a sequence's end: NaN for
    every row of that head (of every head) and for no other."""
    import torch
    hq = 2 * hk
    st = Setup(bk, lens, hk, D, "e4m3", seed=D)
    st.fill()
    q = dev(st.g.standard_normal((sum(new), hq, D)).astype(np.float16))
    good = bk.mq_kv_attention(q, st.cache, st.batch(new))
    assert good.isfinite().all()
    st.cache.k_scale[st.tables[0][3], 1] = float("nan")     # what the append leaves for such a vector
    got = bk.mq_kv_attention(q, st.cache, st.batch(new))
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[:new[0], 2:4] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], good[~bad])
    for missing in (st.cache.num_blocks, -1):
        st.table[1, 4] = missing
        got = bk.mq_kv_attention(q, st.cache, st.batch(new))
        bad[new[0]:] = True
        assert got[bad].isnan().all() and torch.equal(got[~bad], good[~bad])


@pytest.mark.parametrize("new,lens,hq,hk,D", [([1, 1], [2000, 70], 4, 2, 128), ([90, 40], [1500, 700], 4, 2, 64),
                                              ([100], [3000], 4, 2, 128), ([70, 200], [900, 1100], 64, 32, 64)])
def test_attention_under_wide_bounds(bk, new, lens, hq, hk, D):
    """max_new and max_len far above what there is: every row within the tolerance of the oracle."""
    st = Setup(bk, lens, hk, D, "int8", seed=13)
    st.fill()
    q = dev(st.g.standard_normal((sum(new), hq, D)).astype(np.float16))
    b = st.batch(new)
    rows = [0, 1, 31, 39, 64, 89, 99, 128, 199]
    for more, longer in ((1, 8), (3, 1), (5, 30)):
        other = bk.KVBatch(b.cu_q, b.kv_len, b.block_table, b.max_new * more, b.max_len * longer, slots=b.slots)
        check_attention(st, q, new, True, rows=rows, batch=other)
