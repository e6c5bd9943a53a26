"""Every kernel of the head's operators at sizes that use its stages, buffers and segments more than once (head_cases.py says
which size takes which; test_head_plans_cpu.py that it does).

Exact: the products of small whole numbers. Elements are q 2^j with |q| <= 2, j of their block of 128 in 0 .. 2 (tokens) or
0 .. 1 (weights): each is a code, each product at most 2^5 and within 2^2 of the others of its block (so that none is cut),
and with K < 2^15 every sum is a whole number under 2^20, which fp32 holds. So Y is the whole number, rounded once to fp16,
in whatever order it is summed.

Tolerance of the other products: the bound that mosaicq_head.h states, which is that of test_gpu_head.py. Tokens are exact;
log-probabilities of the same row by two kernels are the same bits (whole weights and sums, one logarithm of their quotient).
"""
import math

import numpy as np
import pytest

from oracle import head as oh
from tests import head_cases as hc
from tests.test_gpu_block import SUB, U, close, dev
from tests.test_gpu_head import SETTINGS, halves, hd  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

NAMES = ["-".join(map(str, kernel)) + " %dx%dx%d" % case for case, kernel in hc.LINEAR]


# --------------------------------------------------------------------- product
def whole(seed, shape, most):
    """Float16 whole numbers -2 .. 2 times 2^0 .. 2^most, a power for each block of 128."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-2, 3, shape, generator=g, device="cuda").half()
    j = torch.randint(0, most + 1, (shape[0], -(-shape[1] // 128)), generator=g, device="cuda")
    q *= torch.exp2(j.float()).half().repeat_interleave(128, 1)[:, :shape[1]]
    return q


@pytest.mark.parametrize("case,kernel", hc.LINEAR, ids=NAMES)
def test_products_of_whole_numbers_are_exact(hd, case, kernel):  # noqa: F811
    """Dense tensors, and the same rows inside wider ones, between codes and scales that are NaN."""
    import torch
    M, N, K = case
    x, W = whole(M, (M, K), 2), whole(N + 1, (N, K), 1)
    want = (x.double() @ W.double().t()).half()
    p = hd.mq_pack8(W)
    del W
    codes, scales = hd.mq_quantize8(x)
    got = hd.mq_linear8(codes, scales, p)
    assert torch.equal(got, want), f"{int((got != want).sum())} of {M * N} outputs, the first at {(got != want).nonzero()[0].tolist()}"
    K8, n = codes.shape[1], scales.shape[1]
    wide = torch.full((M, K8 + 144), 127, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + K8] = codes.view(torch.uint8)
    wides = torch.full((M, n + 5), 255, dtype=torch.uint8, device="cuda")
    wides[:, 3:3 + n] = scales.view(torch.uint8)
    out = torch.full((M, N + 9), 7.0, dtype=torch.float16, device="cuda")
    hd.mq_linear8(wide[:, 16:16 + K8].view(torch.float8_e4m3fn), wides[:, 3:3 + n].view(torch.float8_e8m0fnu), p,
                  out=out[:, 5:5 + N])
    assert torch.equal(out[:, 5:5 + N], want)
    assert (out[:, :5] == 7).all() and (out[:, 5 + N:] == 7).all()


GRAPHS = [i for i, (_, k) in enumerate(hc.LINEAR) if k in (("stream", 2, 1), ("tiled", 1, 4, 3), ("tiled", 2, 8, 7), ("tiled", 4, 8, 7))]


@pytest.mark.parametrize("case", [hc.LINEAR[i][0] for i in GRAPHS], ids=[NAMES[i] for i in GRAPHS])
def test_products_in_a_graph(hd, case):  # noqa: F811
    """Kernels that ask for more LDS than a launch has by default, and splits, captured with no call before: every replay
    gives the whole numbers of the codes that it finds."""
    import torch
    M, N, K = case
    W = whole(N, (N, K), 1)
    p, wide = hd.mq_pack8(W), W.double()
    codes, scales = hd.mq_quantize8(whole(0, (M, K), 2))
    ws = torch.empty(max(1, hd.linear8_workspace(p, M)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hd.mq_linear8(codes, scales, p, workspace=ws)
    for seed in (1, 2, 3):
        x = whole(seed, (M, K), 2)
        hd.mq_quantize8(x, codes, scales)
        ws.random_(0, 256)
        graph.replay()
        got = y.clone()
        assert torch.equal(got, (x.double() @ wide.t()).half()), f"replay {seed}"
        assert torch.equal(got, hd.mq_linear8(codes, scales, p))


def bound(want, top, mag, K8):
    """What mosaicq_head.h lets a product be off by."""
    return U * np.abs(want) + SUB + 7 * 2.0 ** -13 * top + 2.0 ** -19 * (K8 / 128 + 1) * mag


def some(n, count, r):
    """The first, the last and some others of n."""
    return np.unique(np.r_[0, n - 1, r.randint(0, n, count)])


@pytest.mark.parametrize("case,kernel", hc.LINEAR, ids=NAMES)
def test_products_of_rows_of_any_size(hd, case, kernel):  # noqa: F811
    """Some outputs of each, against the oracle: scales that differ from block to block, a token and a weight row of NaN."""
    import torch
    M, N, K = case
    g = torch.Generator(device="cuda").manual_seed(M * N)

    def rows(n, spread):
        v = torch.randn((n, K), generator=g, device="cuda")
        v *= torch.exp2(torch.randint(-spread, spread + 1, (n, -(-K // 128)), generator=g, device="cuda").float()
                        ).repeat_interleave(128, 1)[:, :K]
        return v.half()

    x, W = rows(M, 3), rows(N, 2) * 0.0625
    x[M // 2, K - 1], W[N // 3, 0] = math.inf, math.nan
    y = hd.mq_linear8(*hd.mq_quantize8(x), hd.mq_pack8(W))
    nan = torch.isnan(y)
    assert nan[M // 2].all() and nan[:, N // 3].all() and int(nan.sum()) == M + N - 1
    r = np.random.RandomState(M)
    ms, ns = (i[i != skip] for i, skip in ((some(M, 7, r), M // 2), (some(N, 14, r), N // 3)))
    xv, wv = (oh.held(*oh.rows8(t[dev(i)].cpu().numpy())) for t, i in ((x, ms), (W, ns)))
    want, top, mag = oh.linear8(xv, wv)
    close(y[dev(ms)][:, dev(ns)].cpu().numpy(), want, bound(want, top, mag, xv.shape[1]), f"{M} x {N} x {K}")


def product_of(hd, x, W, what):  # noqa: F811
    y = hd.mq_linear8(*hd.mq_quantize8(dev(x)), hd.mq_pack8(dev(W))).cpu().numpy()
    xv, wv = oh.held(*oh.rows8(x)), oh.held(*oh.rows8(W))
    want, top, mag = oh.linear8(xv, wv)
    close(y, want, bound(want, top, mag, xv.shape[1]), what)
    return y, want


@pytest.mark.parametrize("M", [5, 30, 70, 200])
@pytest.mark.parametrize("kind", ["one size", "many sizes", "just under the cut"])
def test_products_of_one_sign(hd, kind, M):  # noqa: F811
    """Cuts that all go the same way. In the last kind seven products of each group of 8 are cut whole."""
    N, K = 20, 5001
    r = np.random.RandomState(M)
    if kind == "just under the cut":
        x, W = np.full((M, K), 2.0), np.full((N, K), 3.75)
        x[:, ::8] = W[:, ::8] = 256.0                     # 2^16, and 7.5 where all under 2^3 is cut
        W *= 2.0 ** -18
    else:
        x, W = (2.0 ** r.uniform(0, 1, s) if kind == "one size" else 2.0 ** r.uniform(-6, 6, s) for s in ((M, K), (N, K)))
        W *= 2.0 ** -8
    y, want = product_of(hd, x.astype(np.float16), W.astype(np.float16), kind)
    assert (np.abs(y - want) <= (7 * 2.0 ** -13 + U + 2.0 ** -19 * 41) * want).all()


@pytest.mark.parametrize("M", [5, 30, 70, 200])
@pytest.mark.parametrize("apart", [1, 4, 1280])
def test_products_that_cancel(hd, M, apart):  # noqa: F811
    """Every product but the last block's comes again with the other sign, in its own group of 8 or in another block."""
    N, K = 20, 2560
    r = np.random.RandomState(M + apart)
    x, W = np.zeros((M, K + 128)), np.zeros((N, K + 128))
    first = np.arange(K).reshape(-1, 2, apart)[:, 0].ravel()
    for t, sign in ((x, 1), (W, -1)):
        t[:, first] = r.randn(len(t), K // 2)
        t[:, first + apart] = sign * t[:, first]
        t[:, K:] = r.randn(len(t), 128) * 2.0 ** -4
    product_of(hd, x.astype(np.float16), W.astype(np.float16), f"{apart} apart")


@pytest.mark.parametrize("M", [1, 40])
def test_the_longest_sums(hd, M):  # noqa: F811
    """K of 2^20, one sign; the first and the last token."""
    import torch
    N, K = 3, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(M)
    x, W = ((1 + torch.rand((n, K), generator=g, device="cuda")).half() for n in (M, N))
    W *= 2.0 ** -14
    y = hd.mq_linear8(*hd.mq_quantize8(x), hd.mq_pack8(W)).cpu().numpy()
    ms = sorted({0, M - 1})
    xv, wv = (oh.held(*oh.rows8(t.cpu().numpy())) for t in (x[ms], W))
    want, top, mag = oh.linear8(xv, wv)
    close(y[ms], want, bound(want, top, mag, K), f"{M} tokens")


@pytest.mark.parametrize("K", [1, 200, 1281])
def test_blocks_that_are_not_finite_are_nan_up_to_their_end(hd, K):  # noqa: F811
    """By the quantizer and by the norm: all codes of such a block are 127, also past the row's end; other blocks are as ever,
    and 0 past the row's end."""
    import torch
    from bit_gemm_amd import block as bk
    x = torch.ones((4, K), device="cuda")
    x[1, K - 1], x[2, 0] = math.inf, math.nan
    n = -(-K // 128)
    for codes, scales in (hd.mq_quantize8(x.half()),
                          bk.mq_norm_residual_q8(None, x, torch.ones(K, dtype=torch.float16, device="cuda"))[1:]):
        c, s = (t.view(torch.uint8).cpu().numpy() for t in (codes, scales))
        assert c.shape == (4, 128 * n) and (c[0, K:] == 0).all() and (c[3, K:] == 0).all() and (s[[0, 3]] == 119).all()
        assert (c[1, 128 * (n - 1):] == 127).all() and s[1, n - 1] == 255
        assert (c[2, :128] == 127).all() and s[2, 0] == 255
        if n > 1:
            assert (c[2, K:] == 0).all() or s[2, n - 1] == 255       # the norm spreads a NaN over its row


# -------------------------------------------------------------------- sampling
def rows_of_settings(R, r):
    pick = r.randint(0, len(SETTINGS), R)
    t, k, p, m = (np.array([SETTINGS[i][j] for i in pick], dt) for j, dt in
                  ((0, np.float32), (1, np.int32), (2, np.float32), (3, np.float32)))
    u = r.rand(R).astype(np.float32)
    u[r.rand(R) < 0.1], u[r.rand(R) < 0.1] = 0.0, 1.0 - 2.0 ** -24
    return u, t, k, p, m


def check(hd, l, settings, some_rows, alone):  # noqa: F811
    """All rows by one call, some against the oracle, all (in turn) against calls of `alone` rows."""
    import torch
    R, V = l.shape
    on = [dev(a) for a in settings]
    token, logprob = hd.mq_sample(l, *on)
    for i in some_rows:
        u, t, k, p, m = (a[i] for a in settings)
        want, lp, kept = oh.sample(l[i].float().cpu().numpy(), u, t, int(k), p, m)
        assert token[i].item() == want, f"row {i}: token {token[i].item()}, want {want} of {len(kept)} kept"
        assert abs(logprob[i].item() - lp) <= 2.0 ** -23 * abs(lp) + 2.0 ** -40 * V
    for a in range(0, R, alone):
        got = hd.mq_sample(l[a:a + alone], *(x[a:a + alone] for x in on))
        assert torch.equal(got[0], token[a:a + alone]) and torch.equal(got[1], logprob[a:a + alone]), f"rows {a} .."


def spread_logits(R, V, dtype, seed):
    """Rows of several kinds: normal of any sharpness, half or almost all of it masked, few values, one narrow step."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((R, V), generator=g, device="cuda")
    l *= torch.exp2(torch.randint(-1, 3, (R, 1), generator=g, device="cuda").float())
    for i in range(1, R, 6):
        l[i, torch.rand(V, generator=g, device="cuda") < 0.5] = -math.inf
    for i in range(2, R, 6):
        l[i, torch.rand(V, generator=g, device="cuda") < 0.999] = -math.inf
        l[i, V - 1] = 0.25
    for i in range(3, R, 6):                   # many equal logits around every limit
        l[i] = torch.randint(-2, 3, (V,), generator=g, device="cuda").float()
    for i in range(4, R, 6):                   # many that differ in their last bits
        l[i] = 1.0 + torch.randint(0, 3000, (V,), generator=g, device="cuda").float() * 2.0 ** -22
    return l.half() if dtype == "float16" else l


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("case,by_rows", hc.SAMPLE, ids=["%dx%d" % c for c, _ in hc.SAMPLE])
def test_sample_on_both_sides_of_the_rules(hd, case, by_rows, dtype):  # noqa: F811
    """Each row the same by a workgroup and over the whole GPU, and as the oracle draws it."""
    R, V = case
    r = np.random.RandomState(R + V)
    alone = next(n for n in (40, 9, 5, 3, 1) if n < R or R == 1)
    if R > 1:
        assert hc.sample_by_rows(alone, V)[0] is False
    few = [0, R - 1, *r.randint(0, R, 5)] if V < 100000 else [3, R - 1]
    check(hd, spread_logits(R, V, dtype, V), rows_of_settings(R, r), sorted(set(few)), alone)


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("R,V", [(64, 20000), (200, 50257), (4, 50257), (2, 262145), (1, 1 << 20)])
def test_sample_where_more_tokens_tie_than_a_list_holds(hd, R, V, dtype):  # noqa: F811
    """Limits by count and by mass that end inside a run of 4000 equal logits and more: found by the search over digits."""
    import torch
    r = np.random.RandomState(V)
    g = torch.Generator(device="cuda").manual_seed(V)
    run = 4000
    l = torch.randn((R, V), generator=g, device="cuda") - 6.0
    for i in range(R):
        at = torch.randperm(V, generator=g, device="cuda")
        l[i, at[:run]] = 1.5
        l[i, at[run:run + 60]] = 2.0 + torch.rand(60, generator=g, device="cuda")
    l = l.half() if dtype == "float16" else l
    k = np.where(np.arange(R) % 3 < 2, r.randint(100, run, R), 0).astype(np.int32)     # inside the run; none
    p = np.where(np.arange(R) % 3 > 0, r.uniform(0.3, 0.8, R), 1.0).astype(np.float32)
    if R == 1:
        k[:], p[:] = 2500, 0.5
    s = (r.rand(R).astype(np.float32), np.ones(R, np.float32), k, p, np.where(np.arange(R) % 2, 0.01, 0).astype(np.float32))
    few = sorted({0, 1 % R, 2 % R, R - 1}) if V <= 262145 else [0]
    check(hd, l, s, few, 40 if R > 40 else 1)


@pytest.mark.parametrize("R,V", [(192, 100003), (192, 262144), (5, 262145)])
def test_sample_draws_from_every_segment(hd, R, V):  # noqa: F811
    """Equal logits: the token is floor(u V), wherever in the row it lies, for a row by a workgroup and over the GPU."""
    import torch
    u = (np.arange(R) / R + 1e-4).astype(np.float32)
    token, logprob = hd.mq_sample(torch.zeros((1, V), dtype=torch.float16, device="cuda").expand(R, V), dev(u))
    want = [int(float(x) * 2 ** 31) * V >> 31 for x in u]       # u counts in steps of 2^-31
    assert token.tolist() == want
    assert torch.allclose(logprob, torch.full_like(logprob, -math.log(V)), rtol=2.0 ** -23, atol=2.0 ** -23)


# --------------------------------------------------------------------- refusals
def test_workspaces_that_are_too_small_are_refused_where_one_is_needed(hd):  # noqa: F811
    import torch
    l = torch.zeros((2, 300000), dtype=torch.float16, device="cuda")
    need = hd.sample_workspace(2, 300000)
    assert need > 0
    with pytest.raises(hd.MQError):
        hd.mq_sample(l, torch.rand(2, device="cuda"), workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    M, N, K = 359, 962, 17050
    p = hd.mq_pack8(dev(halves(1, (N, K), 1)))
    need = hd.linear8_workspace(p, M)
    assert need == 7 * 4 * M * N
    c, s = hd.mq_quantize8(torch.zeros((M, K), dtype=torch.float16, device="cuda"))
    with pytest.raises(hd.MQError):
        hd.mq_linear8(c, s, p, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
