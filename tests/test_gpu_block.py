"""The block operators on the GPU against the float64 oracle (oracle/block.py).

Tolerances, from the operators' definitions (u = 2^-11 for the one rounding to
fp16, e = 2^-24 for an fp32 step, s = 2^-25 for half an fp16 subnormal step):
  rotation   u |y| + s + 5 e m (|a| + |b|): table, two products, a sum
  attention  u |o| + s + (u + 2 d) sum p |v| + L s max |v|: the rounding of p to
             fp16 (relative u, and s for each of L tokens), and the scores'
             error d = (dim + 8) e max scale sum |q| |k| in p and in its sum,
             plus dim + 8 + L / 16 fp32 steps of the sums
  norm       u |h| + s + (width / 64 + 24) e |h|; r' in fp32 with the same steps
codes and scales are exact: the definition's fp32 steps have one result.
"""
import numpy as np
import pytest

from oracle import block as ob

pytestmark = pytest.mark.gpu
U, E, SUB = 2.0 ** -11, 2.0 ** -24, 2.0 ** -25


@pytest.fixture(scope="module")
def bk():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X; none is visible"
    from bit_gemm_amd import block
    return block


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def close(got, want, tol, what):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN at other places"
    with np.errstate(invalid="ignore"):
        bad = np.abs(got - want) > tol
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first {i}: {got[i]!r}, want {want[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, got.shape)[i]!r}")


# ------------------------------------------------------------------- rotary
def rope_tol(x, want, n, layout, mag):
    a = np.abs(np.asarray(x, np.float64))
    pair = a.copy()
    if layout == "half":
        pair[..., :n] = pair[..., n:2 * n] = a[..., :n] + a[..., n:2 * n]
    else:
        pair[..., 0:2 * n:2] = pair[..., 1:2 * n:2] = a[..., 0:2 * n:2] + a[..., 1:2 * n:2]
    return U * np.abs(want) + SUB + 5 * E * mag * pair


ROPES = [  # tokens, heads, dim, rot, layout, scaling, factor, inverse
    (1, 1, 64, 64, "half", "none", 1.0, False),
    (3, 5, 128, 128, "half", "linear", 4.0, False),
    (7, 2, 128, 64, "interleaved", "base", 8.0, True),
    (5, 3, 96, 96, "interleaved", "parts", 8.0, False),
    (4, 3, 80, 32, "half", "parts", 4.0, True),
    (2, 7, 64, 6, "half", "none", 1.0, False),         # a few pairs: element by element
    (2, 3, 33, 10, "interleaved", "none", 1.0, False),  # odd heads
    (300, 33, 256, 256, "half", "none", 1.0, False),
    (1100, 40, 128, 96, "half", "none", 1.0, False),    # enough rows for several heads a thread
    (1101, 41, 128, 128, "interleaved", "none", 1.0, True),
]


@pytest.mark.parametrize("T,H,D,rot,layout,scaling,factor,inverse", ROPES)
def test_rope(bk, T, H, D, rot, layout, scaling, factor, inverse):
    print("rope", T, H, D, rot, layout, scaling, flush=True)
    g = np.random.default_rng(T + D)
    x = (g.standard_normal((T, H, D)) * 3).astype(np.float16)
    positions = 131072 if T < 10 else 3000
    pos = g.integers(0, positions, T).astype(np.int32)
    pos[0] = positions - 1
    f, mag = ob.frequencies(rot, 500000.0, scaling, factor)
    r = bk.Rope(rot, positions, layout=layout, theta=500000.0, scaling=scaling, factor=factor)
    rows = slice(None) if T < 10 else slice(0, T, 17)
    want = ob.rope(x[rows], pos[rows], f, mag, layout, inverse)
    tol = rope_tol(x[rows], want, rot // 2, layout, mag)
    xd, pd = dev(x), dev(pos)
    y = bk.mq_rope(xd, r, pd, inverse=inverse)
    close(y.cpu().numpy()[rows], want, tol, "out")
    z = bk.mq_rope(xd, r, pd, inverse=inverse, out=xd)           # in place
    assert z is xd and (z == y).all()


def test_rope_table_is_rounded_once(bk):
    f, mag = ob.frequencies(128, 10000.0, "parts", 16.0)
    r = bk.Rope(128, 200000, theta=10000.0, scaling="parts", factor=16.0)
    t = r.table.cpu().numpy().astype(np.float64)
    p = np.array([0, 1, 2, 1023, 65536, 131071, 199999])
    for i, fn in ((0, np.cos), (1, np.sin)):
        w = mag * fn(p[:, None] * f[None])
        # one rounding, and the 64-bit angle's own error
        assert np.all(np.abs(t[p, :, i] - w) <= E * np.abs(w) + 1e-10)


def test_rope_strides_and_positions_outside_the_table(bk):
    import torch
    g = np.random.default_rng(5)
    wide = dev(g.standard_normal((6, 3 * 4 * 64 + 5)).astype(np.float16))
    x = wide[:, 5:5 + 4 * 64].unflatten(1, (4, 64))             # rows that are not 16-byte aligned
    r = bk.Rope(64, 50)
    pos = torch.tensor([0, 49, 50, -1, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    y = bk.mq_rope(x, r, pos)
    ok = [0, 1, 5]
    f, _ = ob.frequencies(64)
    xs = x.cpu().numpy()
    want = ob.rope(xs[ok], pos.cpu().numpy()[ok], f)
    close(y.cpu().numpy()[ok], want, rope_tol(xs[ok], want, 32, "half", 1.0), "aligned or not")
    assert y[2:5].isnan().all() and torch.equal(bk.mq_rope(x.contiguous(), r, pos)[:2], y[:2])
    # heads outermost (a transposed view), output into a slice
    xt = x.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.zeros((6, 4, 128), dtype=torch.float16, device="cuda")
    bk.mq_rope(xt, r, pos, out=out[..., :64])
    assert torch.equal(out[:2, :, :64], y[:2]) and not out[..., 64:].any()


def test_rope_gradient_is_the_inverse(bk):
    # <R x, y> = <x, R^T y>, and R is linear: a difference of outputs is the output of the difference
    import torch
    g = np.random.default_rng(6)
    x, y = (dev(g.standard_normal((9, 4, 128)).astype(np.float16)) for _ in range(2))
    pos = torch.arange(0, 9 * 37, 37, dtype=torch.int32, device="cuda")
    for layout in ("half", "interleaved"):
        r = bk.Rope(96, 1000, layout=layout)
        rx, ry = bk.mq_rope(x, r, pos).double(), bk.mq_rope(y, r, pos, inverse=True).double()
        a, b = (rx * y.double()).sum(), (x.double() * ry).sum()
        assert abs(a - b) <= 2 * U * (rx.abs() * y.double().abs()).sum()
        step = 0.25
        diff = (bk.mq_rope(x + step * y, r, pos).double() - bk.mq_rope(x, r, pos).double()) / step
        want = bk.mq_rope(y, r, pos).double()
        assert ((diff - want).abs() <= 4 * U / step * (x.double().abs().max() + y.double().abs().max()) * 2).all()


# -------------------------------------------------------------------- cache
class Setup:
    """A cache on both sides, with blocks scattered over the pool and rubbish
    wherever nothing is written."""

    def __init__(self, bk, lens, hk, D, fmt, seed, extra=2):
        import torch
        self.bk, self.lens, self.hk, self.D, self.fmt = bk, list(lens), hk, D, fmt
        g = np.random.default_rng(seed)
        S = len(lens)
        need = [max(1, -(-n // 64)) for n in lens]
        blocks = sum(need) + extra
        ids = g.permutation(blocks)
        self.tables = [list(ids[sum(need[:s]):sum(need[:s + 1])]) for s in range(S)]
        table = np.full((S, max(need) + 1), -1, np.int32)
        for s, t in enumerate(self.tables):
            table[s, :len(t)] = t
        self.slots = g.permutation(S + 2)[:S].astype(np.int32)
        self.ref = ob.Cache(blocks, S + 2, hk, D, fmt)
        self.cache = bk.KVCache.empty(blocks, S + 2, hk, D, fmt)
        nan = float("nan")
        for c in (self.cache.k_scale, self.cache.v_scale, self.cache.k_tail, self.cache.v_tail):
            c.fill_(nan)
        self.table, self.dslots = dev(table), dev(self.slots)
        self.g = g
        self.torch = torch

    def batch(self, new, lens=None, slots=True):
        lens = self.lens if lens is None else lens
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        return self.bk.KVBatch(dev(cu), dev(np.array(lens, np.int32)), self.table, max(1, max(new)), max(1, max(lens)),
                               slots=self.dslots if slots else None)

    def fill(self, values=None):
        """Every sequence's tokens, in the oracle, and copied to the GPU's cache."""
        for s, n in enumerate(self.lens):
            k, v = ((self.g.standard_normal((n, self.hk, self.D)) * 1.5).astype(np.float16) for _ in range(2))
            if values:
                values(s, k, v)
            self.ref.put(n, self.tables[s], self.slots[s], k, v)
        self.upload()

    def upload(self):
        t = self.torch
        for n in ("k_codes", "v_codes"):
            getattr(self.cache, n).view(t.uint8).copy_(dev(getattr(self.ref, n)))
        for s, n in enumerate(self.lens):
            b = self.tables[s][:n // 64]
            for name in ("k_scale", "v_scale"):
                getattr(self.cache, name)[b] = dev(getattr(self.ref, name)[b]) if b else getattr(self.cache, name)[b]
            o, sl = n % 64, int(self.slots[s])
            if o:
                self.cache.k_tail[sl, :, :o] = dev(self.ref.k_tail[sl, :, :o])
                self.cache.v_tail[sl, :, :, :o] = dev(self.ref.v_tail[sl, :, :, :o])

    def same_cache(self, lens):
        """Codes and scales of full blocks and the open tokens are the oracle's, bit for bit."""
        c = {n: getattr(self.cache, n).view(self.torch.uint8 if "codes" in n else getattr(self.cache, n).dtype).cpu().numpy()
             for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")}
        for s, n in enumerate(lens):
            b, o, sl = self.tables[s][:n // 64], n % 64, int(self.slots[s])
            for name in ("k_scale", "v_scale", "k_codes", "v_codes"):
                assert np.array_equal(c[name][b], getattr(self.ref, name)[b], equal_nan="scale" in name), (name, s)
            assert np.array_equal(c["k_tail"][sl, :, :o], self.ref.k_tail[sl, :, :o], equal_nan=True), ("k_tail", s)
            assert np.array_equal(c["v_tail"][sl, :, :, :o], self.ref.v_tail[sl, :, :, :o]), ("v_tail", s)


APPENDS = [  # lengths of the steps of each sequence, kv heads, dim, format
    ([[1], [64], [65], [63, 1]], 2, 64, "int8"),
    ([[130, 1, 1], [62, 1, 1], [0, 64, 128], [5, 3, 300]], 1, 128, "e4m3"),
    ([[200, 70, 130]], 3, 128, "int8"),                  # steps that start and end inside blocks
    ([[1] * 66, [63] + [1] * 65], 2, 64, "e4m3"),        # token by token through a whole block
    ([[10, 118, 64]], 8, 64, "int8"),
]


@pytest.mark.parametrize("steps,hk,D,fmt", APPENDS)
def test_append_codes_are_exact(bk, steps, hk, D, fmt):
    total = [sum(x) for x in steps]
    st = Setup(bk, total, hk, D, fmt, seed=hk * D)
    lens = [0] * len(steps)
    for i in range(max(len(x) for x in steps)):
        new = [x[i] if i < len(x) else 0 for x in steps]
        lens = [a + b for a, b in zip(lens, new)]
        print("append", new, lens, flush=True)
        T = sum(new)
        # keys and values as slices of one wider row, as a joined projection leaves them
        rows = (st.g.standard_normal((T, (2 * hk + 1) * D + 8)) * 2).astype(np.float16)
        rows[:, ::7] *= 8
        d = dev(rows)
        k, v = d[:, 8:8 + hk * D].unflatten(1, (hk, D)), d[:, 8 + hk * D:8 + 2 * hk * D].unflatten(1, (hk, D))
        at = 0
        for s, n in enumerate(new):
            part = rows[at:at + n, 8:8 + 2 * hk * D].reshape(n, 2, hk, D)
            st.ref.put(lens[s], st.tables[s], st.slots[s], part[:, 0], part[:, 1])
            at += n
        q = bk.mq_kv_append(None, k, v, st.cache, st.batch(new, lens))
        assert q is None
        st.same_cache(lens)
    # nothing else of the pool is written
    used = sorted(b for s, n in enumerate(lens) for b in st.tables[s][:n // 64])
    other = [b for b in range(st.cache.num_blocks) if b not in used]
    assert st.cache.k_scale[other].isnan().all() and not st.cache.v_codes.view(st.torch.uint8)[other].any()


def test_append_extremes(bk):
    """Largest and smallest fp16 values, zeros, and vectors that are not finite."""
    for fmt in ("int8", "e4m3"):
        st = Setup(bk, [128, 70, 64], 2, 64, fmt, seed=3)
        ks, vs = [], []
        for s, n in enumerate(st.lens):
            k, v = (st.g.standard_normal((n, 2, 64)).astype(np.float16) for _ in range(2))
            if s == 0:
                k[:64, 0] *= np.float16(1e-7)             # subnormal
                k[64:, 0] = 0
                v[:, 1] = np.where(v[:, 1] > 0, 65504, -65504)
            if s == 1:
                k[3, 0, 5], v[66, 1, 2], v[65, 1, 3] = np.inf, np.nan, -np.inf
            if s == 2:
                v[63, 0, 0] = np.nan
            ks.append(k)
            vs.append(v)
            st.ref.put(n, st.tables[s], st.slots[s], k, v)
        bk.mq_kv_append(None, dev(np.concatenate(ks)), dev(np.concatenate(vs)), st.cache, st.batch(st.lens))
        st.same_cache(st.lens)


@pytest.mark.parametrize("layout,rot,D,align", [("half", 128, 128, 0), ("interleaved", 64, 64, 0), ("half", 32, 64, 4),
                                                ("interleaved", 6, 128, 0), ("half", 10, 64, 1)])
def test_append_with_rotation(bk, layout, rot, D, align):
    """Queries and keys turned on the way in: the same bits as mq_rope before an append without it."""
    import torch
    hk, hq, new, old = 2, 6, [1, 70, 0, 5], [100, 58, 20, 0]
    st = Setup(bk, [a + b for a, b in zip(new, old)], hk, D, "int8", seed=rot)
    two = Setup(bk, st.lens, hk, D, "int8", seed=rot)
    r = bk.Rope(rot, 200, layout=layout)
    pre = [(st.g.standard_normal((sum(old), hk, D))).astype(np.float16) for _ in range(2)]
    for x in (st, two):
        bk.mq_kv_append(None, dev(pre[0]), dev(pre[1]), x.cache, x.batch(old, old))
    T = sum(new)
    rows = dev(st.g.standard_normal((T, (hq + 2 * hk) * D + align)).astype(np.float16))[:, align:]
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split((hq * D, hk * D, hk * D), 1))
    pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)]).astype(np.int32)
    f, _ = ob.frequencies(rot)
    got = bk.mq_kv_append(q, k, v, st.cache, st.batch(new), rope=r)
    want = ob.rope(q.cpu().numpy(), pos, f, 1.0, layout)
    close(got.cpu().numpy(), want, rope_tol(q.cpu().numpy(), want, rot // 2, layout, 1.0), "queries")
    assert torch.equal(got, bk.mq_rope(q, r, dev(pos)))
    bk.mq_kv_append(None, bk.mq_rope(k, r, dev(pos)), v, two.cache, two.batch(new))
    for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
        a, b = (getattr(x.cache, n) for x in (st, two))
        a, b = (x.view(torch.uint8) if "codes" in n else x for x in (a, b))
        assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a, b.nan_to_num(7.0) if b.is_floating_point() else b), n
    # in place, and the same step again gives the same cache
    before = st.cache.k_tail.clone()
    bk.mq_kv_append(q, k, v, st.cache, st.batch(new), rope=r, q_out=q)
    assert torch.equal(q, got)
    assert torch.equal(before[st.slots[0]].nan_to_num(), st.cache.k_tail[st.slots[0]].nan_to_num())


def test_append_drops_what_has_no_place(bk):
    """Blocks and slots out of range, lengths past the table: nothing is written there, the rest is."""
    import torch
    st = Setup(bk, [128, 128, 30], 2, 64, "int8", seed=9)
    st.table[0, 1] = 10 ** 6
    st.dslots[2] = -5
    g = np.random.default_rng(1)
    k, v = (g.standard_normal((286, 2, 64)).astype(np.float16) for _ in range(2))
    b = st.batch([128, 128, 30])
    bk.mq_kv_append(None, dev(k), dev(v), st.cache, b)
    torch.cuda.synchronize()
    c, s = ob.quantise(k[:64, 0], "int8")
    assert np.array_equal(st.cache.k_codes[st.tables[0][0], 0].cpu().numpy().view(np.uint8), c)
    assert np.array_equal(st.cache.k_codes[st.tables[1][1], 0].cpu().numpy().view(np.uint8), ob.quantise(k[192:256, 0], "int8")[0])
    assert st.cache.k_scale[st.tables[0][1]].isnan().all() and st.cache.k_tail.isnan().all()
    # a sequence longer than its table
    far = bk.KVBatch(dev(np.array([0, 64], np.int32)), dev(np.array([10000], np.int32)), st.table[:1], 64, 10000)
    bk.mq_kv_append(None, dev(k[:64]), dev(v[:64]), st.cache, far)
    torch.cuda.synchronize()
    assert st.cache.k_tail.isnan().all()


# ---------------------------------------------------------------- attention
def check_attention(st, q, new, causal, scale=None, what="", rows=None, lens=None, batch=None):
    D, hk = st.D, st.hk
    lens = st.lens if lens is None else lens
    hq = q.shape[1]
    scale = D ** -0.5 if scale is None else scale
    qn = q.cpu().numpy().astype(np.float64)
    batch = batch or st.batch(new, lens)
    got = st.bk.mq_kv_attention(q, st.cache, batch, causal=causal, scale=scale).cpu().numpy()
    at = 0
    for s, n in enumerate(new):
        L = lens[s]
        for h in range(hk):
            k, v = st.ref.read(L, st.tables[s], st.slots[s], h)
            vmax = np.abs(v[np.isfinite(v)]).max() if L else 0.0
            for i in range(n) if rows is None else [x for x in rows if x < n]:
                vis = L - n + i + 1 if causal else L
                for hh in range(h * hq // hk, (h + 1) * hq // hk):
                    o, pv, sa = ob.attend(qn[at + i, hh], k, v, vis, scale)
                    d = (D + 8) * E * sa
                    tol = U * np.abs(o) + SUB + (U + 2 * d + (D + 8 + L / 16) * E) * pv + max(vis, 0) * SUB * vmax
                    close(got[at + i, hh], o, tol, f"{what} seq {s} token {i} head {hh}")
        at += n
    return got


ATTENTIONS = [  # new tokens, lengths, query heads, kv heads, dim, causal
    ([1], [1], 1, 1, 64, True),
    ([1, 1, 1, 1, 1], [1, 63, 64, 65, 129], 4, 2, 128, True),
    ([1], [3000], 2, 1, 128, True),                     # split over the cache
    ([1, 1], [2500, 90], 16, 1, 64, True),
    ([1], [700], 5, 1, 128, False),                     # an odd group
    ([1, 0, 3, 16], [200, 77, 3, 300], 8, 2, 64, True),  # ragged, one sequence without new tokens
    ([7, 2], [500, 2], 8, 2, 128, True),                # 28 rows a kv head
    ([5], [130], 71, 71, 64, False),
    ([20], [85], 3, 3, 128, False),
    ([100, 33], [100, 333], 4, 1, 128, True),           # prompts
    ([67], [200], 6, 2, 64, True),
    ([130, 1], [1100, 400], 8, 1, 64, True),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,lens,hq,hk,D,causal", ATTENTIONS)
def test_attention(bk, new, lens, hq, hk, D, causal, fmt):
    print("attention", new, lens, hq, hk, D, causal, fmt, flush=True)
    st = Setup(bk, lens, hk, D, fmt, seed=sum(lens) + D)
    st.fill()
    q = dev((st.g.standard_normal((sum(new), hq, D)) * 1.5).astype(np.float16))
    check_attention(st, q, new, causal)


PIECES = [  # many rows: new tokens, lengths, query heads, kv heads, dim, causal; rows that are checked
    ([700], [700], 4, 1, 128, True),
    ([513, 7], [2600, 90], 8, 2, 64, True),
    ([300], [5000], 2, 2, 128, False),                  # the cache split over workgroups
    ([64, 400, 129], [64, 464, 3000], 4, 2, 128, True),
    ([1000], [1024], 1, 1, 64, True),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,lens,hq,hk,D,causal", PIECES)
def test_attention_of_long_pieces(bk, new, lens, hq, hk, D, causal, fmt):
    print("pieces", new, lens, hq, hk, D, causal, fmt, flush=True)
    st = Setup(bk, lens, hk, D, fmt, seed=sum(new) + D)
    st.fill()
    q = dev((st.g.standard_normal((sum(new), hq, D)) * 1.5).astype(np.float16))
    rows = sorted({0, 1, 31, 32, 62, 63, 64, 65, 127, 128, 129, 255, 256, 299, 300, 399, 511, 512, 640, 698, 699, 999})
    check_attention(st, q, new, causal, rows=rows)


def ragged(seed, seqs, hi, longest, empty=0.2):
    """New tokens and lengths of a ragged batch: sequences without new tokens, without a past, longer than 15 blocks."""
    g = np.random.default_rng(seed)
    new = [0 if g.random() < empty else int(g.integers(1, hi + 1)) for _ in range(seqs)]
    new[seqs // 2] = hi
    lens = [n + (0 if g.random() < 0.3 else int(g.integers(0, longest - n))) for n in new]
    lens[-1] = longest
    return new, lens


SLICES = [  # batch, query heads, kv heads, dim, causal: many row tiles, but not enough to fill the GPU twice
    (ragged(1, 20, 150, 1100), 16, 16, 64, True),
    (ragged(2, 20, 150, 1100), 16, 16, 64, False),
    (ragged(3, 9, 160, 1300), 32, 16, 128, True),
    (ragged(4, 9, 160, 1300), 16, 16, 128, False),
    (ragged(5, 130, 90, 1000, 0.5), 3, 3, 64, True),    # more sequences than a wave has lanes
    (([0, 0, 700, 0], [0, 100, 4000, 64]), 48, 24, 64, True),
    (([300], [2000]), 99, 99, 64, True),
    (([520, 260, 1], [520, 2050, 1]), 25, 25, 128, True),
    (([0] * 40 + [65] + [0] * 30, [64] * 40 + [16000] + [0] * 30), 4, 4, 64, True),     # a tile over many slices,
    (([0] * 40 + [257] + [0] * 30, [64] * 40 + [9000] + [0] * 30), 2, 2, 128, True),    # its last row alone in a wave
]


def in_slices(bk, st, b, tokens, hq):
    """Whether the call lays its work out in slices: the size of its workspace is that of no split."""
    rows = 128 if st.D == 64 else 256
    return bk.kv_attention_workspace(st.cache, b, tokens, hq) == 65536 // rows * (2 * rows * (4 * st.D + 8) + 24)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("batch,hq,hk,D,causal", SLICES)
def test_attention_in_slices(bk, batch, hq, hk, D, causal, fmt):
    import torch
    new, lens = batch
    print("slices", new, lens, hq, hk, D, causal, fmt, flush=True)
    st = Setup(bk, lens, hk, D, fmt, seed=sum(new) + D)
    st.fill()
    q = dev((st.g.standard_normal((sum(new), hq, D)) * 1.5).astype(np.float16))
    b = st.batch(new)
    assert in_slices(bk, st, b, len(q), hq)
    got = check_attention(st, q, new, causal, rows=[0, 1, 31, 63, 64, 89, 127, 128, 149, 159, 256, 259, 299, 519, 699])
    # what was in the workspace before does not matter, and the same call gives the same bits
    ws = torch.full((bk.kv_attention_workspace(st.cache, b, len(q), hq),), 255, dtype=torch.uint8, device="cuda")
    again = bk.mq_kv_attention(q, st.cache, b, causal=causal, workspace=ws).cpu().numpy()
    assert np.array_equal(got.view(np.int16), again.view(np.int16))


def test_slices_of_rows_with_nothing_to_see(bk):
    """Sequences that are empty, or have more new tokens than tokens, among others: zeros where nothing is seen."""
    new, lens = [130, 40, 129, 0, 200, 5], [0, 20, 1000, 7, 100, 5]
    st = Setup(bk, lens, 24, 64, "int8", seed=3)
    st.fill()
    q = dev(st.g.standard_normal((sum(new), 48, 64)).astype(np.float16))
    assert in_slices(bk, st, st.batch(new), len(q), 48)
    got = check_attention(st, q, new, True, rows=[0, 19, 20, 39, 99, 100, 128, 129, 199])
    assert not got[:130].any() and not got[130:150].any() and got[150:170].any(axis=-1).all()


def test_slices_in_a_graph(bk):
    """A captured call follows the lengths and the new tokens that it finds."""
    import torch
    new, lens, hq = [120, 60, 200, 20], [900, 1200, 500, 1030], 64
    st = Setup(bk, lens, 32, 64, "e4m3", seed=8)
    st.fill()
    q = dev(st.g.standard_normal((sum(new), hq, 64)).astype(np.float16))
    b = st.batch(new)
    assert in_slices(bk, st, b, len(q), hq)
    ws = torch.empty(bk.kv_attention_workspace(st.cache, b, len(q), hq), dtype=torch.uint8, device="cuda")
    bk.mq_kv_attention(q, st.cache, b, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = bk.mq_kv_attention(q, st.cache, b, workspace=ws)
    for n, L in ((new, lens), ([0, 200, 0, 200], [0, 1200, 64, 1030]), ([100, 100, 100, 100], [128, 640, 128, 960]),
                 ([1, 199, 199, 1], [64, 256, 448, 1030]), (new, lens)):
        b.cu_q.copy_(torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32))
        b.kv_len.copy_(torch.tensor(L, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = bk.mq_kv_attention(q, st.cache, b)
        assert torch.equal(o.view(torch.int16), eager.view(torch.int16)), (n, L)
        check_attention(st, q, n, True, rows=[0, 63, 99, 128, 198, 199], lens=L, batch=b)


@pytest.mark.parametrize("new,hq", [([2], 4), ([90], 4)])
def test_attention_of_blocks_with_very_different_scales(bk, new, hq):
    """Values of a block that are all zero, or a thousand times another's; keys likewise; negative and zero scales of
    the scores: nothing is lost between blocks."""
    for fmt in ("int8", "e4m3"):
        st = Setup(bk, [500], 1, 128, fmt, seed=11)

        def values(s, k, v):
            v[64:128] = 0
            v[128:192] *= np.float16(1e-3)
            v[192:256] *= np.float16(1e3)
            k[128:256] *= np.float16(1e-2)
            k[256:320] = 0
            v[320:384] *= np.float16(2e-4)
        st.fill(values)
        q = dev(st.g.standard_normal((new[0], hq, 128)).astype(np.float16))
        rows = [0, 1, 40, 63, 89]
        for scale in (128 ** -0.5, -0.5, 0.0):
            check_attention(st, q, new, True, scale=scale, what=f"{fmt} scale {scale}", rows=rows)


@pytest.mark.parametrize("new,lens,D", [([1, 1], [2000, 70], 128), ([90, 40], [1500, 700], 64), ([100], [3000], 128)])
def test_attention_does_not_depend_on_the_bounds(bk, new, lens, D):
    """max_new and max_len choose how the work is split, not what it gives; the same call gives the same bits."""
    import torch
    st = Setup(bk, lens, 2, D, "int8", seed=12)
    st.fill()
    q = dev(st.g.standard_normal((sum(new), 4, D)).astype(np.float16))
    b = st.batch(new)
    want = bk.mq_kv_attention(q, st.cache, b)
    assert torch.equal(want, bk.mq_kv_attention(q, st.cache, b))
    for more, longer in ((1, 8), (3, 1), (5, 30)):
        other = bk.KVBatch(b.cu_q, b.kv_len, b.block_table, b.max_new * more, b.max_len * longer, slots=b.slots)
        got = bk.mq_kv_attention(q, st.cache, other)
        # each is within its own tolerance of the same value: two roundings to fp16 and two of p
        assert ((got - want).abs().double() <= 2 * U * want.abs().double() + 2 * U * 1.5 * 6).all()


def test_attention_rows_with_nothing_to_see(bk):
    """Empty sequences and sequences with more new tokens than tokens: zeros, not NaN."""
    st = Setup(bk, [0, 2, 70], 2, 64, "int8", seed=1)
    st.fill()
    q = dev(st.g.standard_normal((3 + 5 + 2, 4, 64)).astype(np.float16))
    got = check_attention(st, q, [3, 5, 2], True)
    assert not got[:3].any() and not got[3:6].any() and got[6:].all(axis=-1).any()
    assert not check_attention(st, q, [3, 5, 2], False)[:3].any()


def test_attention_of_large_and_small_scores(bk):
    """Scores far apart and far from zero, a scale of 0, a negative one: the maximum is taken out."""
    st = Setup(bk, [300], 1, 64, "int8", seed=2)

    def values(s, k, v):
        k[17] *= np.float16(40)
        k[200:] *= np.float16(1e-4)
    st.fill(values)
    q = dev((st.g.standard_normal((2, 4, 64)) * 8).astype(np.float16))
    for scale in (0.125, 2.0, 0.0, -1.0):
        check_attention(st, q, [2], True, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("new,hq", [([1, 1], 4), ([80, 90], 4)])
def test_attention_with_vectors_that_are_not_finite(bk, new, hq):
    """A bad vector in the open block makes NaN what attends to it, and nothing else; in a coded block every row of
    its head that reads the block; rubbish past a sequence's end or in blocks of others does not count."""
    lens, hk, D = [150, 250], 2, 64
    st = Setup(bk, lens, hk, D, "int8", seed=4)

    def values(s, k, v):
        if s == 0:
            v[148, 0, 3], k[149, 1, 0] = np.nan, np.inf
        else:
            k[130, 1, 2] = np.nan
    st.fill(values)
    q = dev(st.g.standard_normal((sum(new), hq, D)).astype(np.float16))
    got = st.bk.mq_kv_attention(q, st.cache, st.batch(new), causal=True).isnan().cpu().numpy()
    at = 0
    for s, n in enumerate(new):
        for i in range(n):
            p = lens[s] - n + i
            want = [p >= 148, p >= 149] if s == 0 else [False, p >= 128]
            for h in range(hk):
                assert (got[at + i, 2 * h:2 * h + 2] == want[h]).all(), (s, i, h)
        at += n
    # a NaN query is its own row's alone (head 1 of sequence 1's first token; heads 0 and 1 share a kv head without a mark)
    q[new[0], 1] = float("nan")
    again = st.bk.mq_kv_attention(q, st.cache, st.batch(new), causal=True).isnan().cpu().numpy()
    got[new[0], 1] = True
    assert np.array_equal(again, got)


def test_attention_with_tables_out_of_range(bk):
    """A block or slot that does not exist makes NaN of the rows that need it, and of no others."""
    st = Setup(bk, [300, 100], 2, 64, "int8", seed=5)
    st.fill()
    q = dev(st.g.standard_normal((2, 4, 64)).astype(np.float16))
    good = bk.mq_kv_attention(q, st.cache, st.batch([1, 1]))
    st.table[0, 2] = st.cache.num_blocks
    bad = bk.mq_kv_attention(q, st.cache, st.batch([1, 1]))
    assert bad[0].isnan().all() and (bad[1] == good[1]).all()
    st.table[0, 2] = -7
    st.dslots[1] = 99
    bad = bk.mq_kv_attention(q, st.cache, st.batch([1, 1]))
    assert bad.isnan().all()


def test_attention_strides_streams_and_graphs(bk):
    """q and out as slices, another stream, a graph replayed over lengths that grow, the same bits each time."""
    import torch
    hk, hq, D = 2, 8, 128
    st = Setup(bk, [600, 1700], hk, D, "e4m3", seed=6)
    st.fill()
    wide = dev(st.g.standard_normal((2, (hq + 2) * D)).astype(np.float16))
    q = wide[:, D:D + hq * D].unflatten(1, (hq, D))
    b = st.batch([1, 1])
    want = bk.mq_kv_attention(q.contiguous(), st.cache, b)
    out = torch.full((2, hq + 1, D), 5.0, dtype=torch.float16, device="cuda")
    bk.mq_kv_attention(q, st.cache, b, out=out[:, 1:])
    assert torch.equal(out[:, 1:], want) and (out[:, 0] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bk.mq_kv_attention(q, st.cache, b, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(bk.kv_attention_workspace(st.cache, b, 2, hq), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    with pytest.raises(bk.MQError):
        bk.mq_kv_attention(q, st.cache, b, workspace=ws[:-16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = bk.mq_kv_attention(q, st.cache, b, workspace=ws)
    for lens in ([600, 1700], [1, 64], [300, 1650], [600, 1700]):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = bk.mq_kv_attention(q, st.cache, b)
        assert torch.equal(o.view(torch.int16), eager.view(torch.int16)), lens


def test_step_in_a_graph(bk):
    """A decode step (append with rotation, attention) captured once, replayed as sequences grow."""
    import torch
    hk, hq, D = 2, 4, 64
    lens = [60, 190]
    one, two = Setup(bk, [80, 220], hk, D, "int8", seed=7), Setup(bk, [80, 220], hk, D, "int8", seed=7)
    r = bk.Rope(D, 300)
    k0, v0 = (dev(one.g.standard_normal((sum(lens), hk, D)).astype(np.float16)) for _ in range(2))
    for x in (one, two):
        bk.mq_kv_append(None, k0, v0, x.cache, x.batch(lens, lens))
    qkv = torch.zeros((2, hq + 2 * hk, D), dtype=torch.float16, device="cuda")

    def step(x, b):
        q = bk.mq_kv_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], x.cache, b, rope=r)
        return bk.mq_kv_attention(q, x.cache, b)

    b1, b2 = one.batch([1, 1], [80, 220]), two.batch([1, 1], [80, 220])
    b1.kv_len.copy_(dev(np.array(lens, np.int32) + 1))
    step(one, b1)                                       # eager once before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(one, b1)
    for i in range(1, 12):
        qkv.copy_(dev(one.g.standard_normal(tuple(qkv.shape)).astype(np.float16)))
        now = dev(np.array(lens, np.int32) + i)
        b1.kv_len.copy_(now)
        b2.kv_len.copy_(now)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, step(two, b2)), i
    for n in ("k_codes", "v_codes", "k_tail", "v_tail"):
        a, b = (getattr(x.cache, n).view(torch.uint8) for x in (one, two))
        assert torch.equal(a, b), n


def test_cache_past_32_bits(bk):
    """Codes beyond 4 GiB of either array: the last blocks of a pool of that size."""
    import torch
    hk, D, blocks = 8, 128, 65536 + 40                  # 8 x 64 x 128 bytes a block: more than 2^32 in all
    assert blocks * hk * 64 * D > 1 << 32
    k, v = (torch.empty(blocks * hk * 64 * D, dtype=torch.int8, device="cuda") for _ in range(2))
    sc = [torch.zeros((blocks, hk), device="cuda") for _ in range(2)]
    tails = [torch.zeros((1, hk, *s), dtype=torch.float16, device="cuda") for s in ((64, D), (D, 64))]
    big = bk.KVCache(k.view(blocks, hk, 64, D), v.view(blocks, hk, D, 64), *sc, *tails)
    st = Setup(bk, [200], hk, D, "int8", seed=8)
    table = torch.tensor([[blocks - 1, 3, blocks - 2, blocks - 7]], dtype=torch.int32, device="cuda")
    kk, vv = (st.g.standard_normal((200, hk, D)).astype(np.float16) for _ in range(2))
    st.ref.put(200, st.tables[0], st.slots[0], kk, vv)
    st.upload()
    b = bk.KVBatch(dev(np.array([0, 200], np.int32)), dev(np.array([200], np.int32)), table, 200, 200)
    bk.mq_kv_append(None, dev(kk), dev(vv), big, b)
    q = dev(st.g.standard_normal((200, hk, D)).astype(np.float16))
    want = bk.mq_kv_attention(q, st.cache, st.batch([200]))
    assert torch.equal(bk.mq_kv_attention(q, big, b), want)


# -------------------------------------------------------------------- norms
NORMS = [  # tokens, width, post, gate, fp32 residual, alpha, beta, offset
    (1, 1, True, None, False, 1.0, 1.0, 0.0),
    (3, 7, False, "token", True, 0.5, 2.0, 1.0),
    (16, 4096, True, None, False, 1.0, 1.0, 0.0),
    (5, 2048, True, "channel", True, 1.0, 0.22, 1.0),
    (2, 4097, True, "token", False, 1.0, 1.0, 0.0),
    (3, 8192, False, None, False, 1.0, 1.0, 0.0),
    (2, 16384, True, "channel", True, 0.7, -1.0, 0.0),
    (2, 30000, True, "token", True, 1.0, 1.0, 0.0),
    (1, 65536, True, None, False, 1.0, 1.0, 0.0),
    (700, 5120, True, "token", True, 1.0, 1.0, 1.0),
]


@pytest.mark.parametrize("T,W,post,gate,f32,alpha,beta,offset", NORMS)
def test_norm(bk, T, W, post, gate, f32, alpha, beta, offset):
    print("norm", T, W, post, gate, f32, flush=True)
    g = np.random.default_rng(T + W)
    y = (g.standard_normal((T, W)) * 2).astype(np.float16)
    r = (g.standard_normal((T, W)) * 3).astype(np.float32 if f32 else np.float16)
    wp, wq = ((1 - offset + 0.2 * g.standard_normal(W)).astype(np.float16) for _ in range(2))
    wq = wq if post else None
    ga = {None: None, "channel": g.random(W).astype(np.float16), "token": g.random((T, W)).astype(np.float16)}[gate]
    out, mag, h = ob.norm_residual(y, r, wp, wq, ga, alpha, beta, 1e-6, offset)
    steps = (W / 64 + 24) * E
    args = dict(w_post=None if wq is None else dev(wq), gate=None if ga is None else dev(ga), alpha=alpha, beta=beta,
                weight_offset=offset)
    rd = dev(r)
    r2, h2 = bk.mq_norm_residual(dev(y), rd, dev(wp), **args)
    rn = r2.cpu().numpy()
    close(rn, out, steps * mag + (0 if f32 else U * np.abs(out) + SUB), "residual")
    want = h(rn)
    close(h2.cpu().numpy(), want, (U + steps) * np.abs(want) + SUB, "h")
    # in place, rows apart and not aligned, and its parts on their own
    import torch
    big = torch.zeros((T, 2 * W + 3), dtype=torch.float16, device="cuda")
    big[:, 1:W + 1] = dev(y)
    r3, h3 = bk.mq_norm_residual(big[:, 1:W + 1], rd, dev(wp), r_out=rd, h_out=big[:, W + 2:2 * W + 2], **args)
    assert r3 is rd and torch.equal(r3, r2)
    close(h3.cpu().numpy(), want, (U + steps) * np.abs(want) + SUB, "h, unaligned")
    only, none = bk.mq_norm_residual(dev(y), dev(r), None, **args)
    assert none is None and torch.equal(only, r2)
    same, h4 = bk.mq_norm_residual(None, r2, dev(wp), weight_offset=offset)
    assert same is r2
    close(h4.cpu().numpy(), want, (U + steps) * np.abs(want) + SUB, "norm alone")


def test_norm_of_zero_rows_and_large_values(bk):
    import torch
    W = 512
    w = torch.ones(W, dtype=torch.float16, device="cuda")
    z = torch.zeros((2, W), dtype=torch.float16, device="cuda")
    r, h = bk.mq_norm_residual(z, z, w, w_post=w)
    assert not r.any() and not h.any()                       # eps keeps 0 / 0 out
    big = torch.full((1, W), 60000.0, dtype=torch.float16, device="cuda")
    r, h = bk.mq_norm_residual(None, big, w)
    assert (h - 1).abs().max() <= 2 * U                      # squares are summed in fp32, not fp16
    r, h = bk.mq_norm_residual(torch.empty((0, W), dtype=torch.float16, device="cuda"), z[:0], w)
    assert h.shape == (0, W)
