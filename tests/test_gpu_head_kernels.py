"""Every kernel of the head's product at sizes that use its stages, buffers and segments more than once (head_cases.py says
which size takes which; test_head_plans_cpu.py that it does).

Exact: the products of small whole numbers. Elements are q 2^j with |q| <= 2, j of their block of 128 in 0 .. 2 (tokens) or
0 .. 1 (weights): each is a code, each product at most 2^5 and within 2^2 of the others of its block (so that none is cut),
and with K < 2^15 every sum is a whole number under 2^20, which fp32 holds. So Y is the whole number, rounded once to fp16,
in whatever order it is summed.

Tolerance of the other products as in test_gpu_head.py.
"""
import math

import numpy as np
import pytest

from oracle import head as oh
from tests import head_cases as hc
from tests.test_gpu_block import SUB, U, close, dev
from tests.test_gpu_head import halves, hd  # noqa: F401  (the fixture)

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
    tol = U * np.abs(want) + SUB + 7 * 2.0 ** -13 * top + (16 * xv.shape[1] / 128 + 16) * 2.0 ** -23 * mag
    close(y[dev(ms)][:, dev(ns)].cpu().numpy(), want, tol, f"{M} x {N} x {K}")


# --------------------------------------------------------------------- refusals
def test_a_workspace_that_is_too_small_is_refused(hd):  # noqa: F811
    import torch
    M, N, K = 359, 962, 17050
    p = hd.mq_pack8(dev(halves(1, (N, K), 1)))
    need = hd.linear8_workspace(p, M)
    assert need == 7 * 4 * M * N
    c, s = hd.mq_quantize8(torch.zeros((M, K), dtype=torch.float16, device="cuda"))
    with pytest.raises(hd.MQError):
        hd.mq_linear8(c, s, p, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
