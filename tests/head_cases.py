"""Sizes at which the head's operators take each of their kernels. What they take is checked without a GPU
(test_head_plans_cpu.py); the results are checked on one (test_gpu_head_kernels.py)."""
import ctypes
import os

HC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemm_amd", "libmq_hostcheck.so")

# mq_linear8: (tokens, N, K) and the kernel: ("stream", blocks of 16 tokens, blocks of 16 weight rows a workgroup) or
# ("tiled", blocks of 16 weight rows a wave, blocks of 16 tokens, splits along K). Odd N and K; K of 11 blocks of 128 and
# more, so that stages, weight sets and scale buffers are all used again.
LINEAR = [
    ((13, 201, 6200), ("stream", 1, 1)),
    ((16, 33, 20000), ("stream", 1, 1)),
    ((7, 32787, 4900), ("stream", 1, 2)),
    ((29, 203, 6200), ("stream", 2, 1)),
    ((23, 4279, 9001), ("stream", 2, 2)),
    ((38, 1001, 1401), ("tiled", 1, 2, 1)),
    ((47, 9, 7217), ("tiled", 1, 2, 8)),
    ((77, 65, 20001), ("tiled", 1, 2, 8)),
    ((1105, 137, 10782), ("tiled", 1, 2, 2)),
    ((2125, 401, 1402), ("tiled", 1, 4, 1)),
    ((735, 406, 13040), ("tiled", 1, 4, 3)),
    ((414, 571, 32306), ("tiled", 1, 4, 4)),
    ((2062, 201, 1371), ("tiled", 2, 2, 1)),
    ((2338, 73, 10593), ("tiled", 2, 2, 3)),
    ((80, 778, 30224), ("tiled", 2, 2, 8)),
    ((1634, 647, 1359), ("tiled", 2, 4, 1)),
    ((1572, 545, 10931), ("tiled", 2, 4, 2)),
    ((1039, 69, 8043), ("tiled", 2, 4, 8)),
    ((2089, 970, 1369), ("tiled", 2, 8, 1)),
    ((333, 10007, 2501), ("tiled", 2, 8, 1)),
    ((359, 962, 17050), ("tiled", 2, 8, 7)),
    ((194, 16387, 1281), ("tiled", 4, 8, 1)),
    ((194, 16395, 2690), ("tiled", 4, 8, 1)),
    ((1831, 2227, 1353), ("tiled", 4, 8, 1)),
    ((1845, 1035, 9064), ("tiled", 4, 8, 3)),
    ((2063, 450, 14189), ("tiled", 4, 8, 7)),
]

# mq_sample: (rows, vocab), and whether a workgroup takes a row; both sides of each border
SAMPLE = [
    ((1, 16384), True), ((1, 16385), False), ((64, 20000), True), ((64, 20480), True), ((64, 20481), False),
    ((100, 32000), True), ((191, 61120), True), ((191, 61121), False), ((200, 50257), True), ((192, 262144), True),
    ((192, 262145), False),
]


def _lib():
    assert os.path.exists(HC), "libmq_hostcheck.so is not built"
    h = ctypes.CDLL(HC)
    i64, ints = ctypes.c_int64, ctypes.POINTER(ctypes.c_int)
    h.mqh_linear8_plan.argtypes, h.mqh_linear8_plan.restype = [i64, i64, i64, ints], i64
    h.mqh_sample_by_rows.argtypes, h.mqh_sample_by_rows.restype = [i64, i64, ints, ints], ctypes.c_int
    return h


def linear_kernel(M, N, K):
    """The kernel that a product takes, as in LINEAR, and its bytes of workspace."""
    plan = (ctypes.c_int * 6)()
    n = _lib().mqh_linear8_plan(M, N, K, plan)
    nt, r, _, tb, splits, _ = plan
    return (("stream", nt, r) if nt else ("tiled", r, tb, splits)), n


def sample_by_rows(rows, vocab):
    """Whether a workgroup takes a row; a row's workgroups and the tokens of a segment where not."""
    splits, span = ctypes.c_int(), ctypes.c_int()
    by_rows = bool(_lib().mqh_sample_by_rows(rows, vocab, ctypes.byref(splits), ctypes.byref(span)))
    return by_rows, splits.value, span.value
