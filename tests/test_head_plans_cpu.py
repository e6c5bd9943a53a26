"""The sizes that the GPU tests of the head's kernels use reach the kernels that they name: the rules of head_plan.h, built
for the host, and the workspaces that the library states."""
import ctypes

import pytest

from tests import head_cases as hc
from tests.test_head_abi_cpu import _w8, hd  # noqa: F401  (the fixture)


@pytest.mark.parametrize("case,kernel", hc.LINEAR)
def test_linear_kernels(hd, case, kernel):  # noqa: F811
    M, N, K = case
    got, ws = hc.linear_kernel(M, N, K)
    assert got == kernel
    n = ctypes.c_size_t()
    assert hd.lib.mq_linear8_workspace(M, ctypes.byref(_w8(hd, N=N, K=K)), ctypes.byref(n)) == 0
    assert n.value == ws == (4 * M * N * kernel[3] if kernel[0] == "tiled" and kernel[3] > 1 else 0)


def test_every_linear_kernel_is_among_them():
    kernels = {k for _, k in hc.LINEAR}
    assert {k for k in kernels if k[0] == "stream"} == {("stream", nt, r) for nt in (1, 2) for r in (1, 2)}
    for r, tb in ((1, 2), (1, 4), (2, 2), (2, 4), (2, 8), (4, 8)):
        splits = {k[3] for k in kernels if k[:3] == ("tiled", r, tb)}
        assert 1 in splits and max(splits) > 1, (r, tb)
    # the shapes that the rule can choose at all
    import random
    rng = random.Random(1)
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(0, top)) for top in (12, 16, 16))
        k, _ = hc.linear_kernel(M, N, K)
        assert k[:3] in {x[:3] for x in kernels}, (M, N, K, k)
    for (_, N, K), k in hc.LINEAR:
        assert N % 4 and -(-K // 128) >= 11


@pytest.mark.parametrize("case,by_rows", hc.SAMPLE)
def test_sample_kernels(hd, case, by_rows):  # noqa: F811
    got, splits, span = hc.sample_by_rows(*case)
    assert got == by_rows
    a, n = hd._SampleArgs(rows=case[0], vocab=case[1]), ctypes.c_size_t()
    assert hd.lib.mq_sample_workspace(ctypes.byref(a), ctypes.byref(n)) == 0
    assert (n.value == 0) == by_rows
    assert splits <= 64 and 8 * splits * span >= case[1]
