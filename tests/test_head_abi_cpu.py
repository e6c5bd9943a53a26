"""C ABI of the head's operators, without a GPU: the library exports exactly what include/mosaicq_head.h declares and
refuses bad arguments before any HIP call; so does mq_norm_residual_q8."""
import ctypes
import os
import re
import subprocess

import pytest

from tests.test_block_abi_cpu import bk  # noqa: F401  (the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_gemm_amd", "libmosaicq_head.so")
HEADER = os.path.join(ROOT, "include", "mosaicq_head.h")
A = 1 << 20                     # an aligned address that validation never reads
BAD, UNS = -1, -2


@pytest.fixture(scope="module")
def hd():
    assert os.path.exists(LIB), "libmosaicq_head.so is not built (python -m bit_gemm_amd.build)"
    from bit_gemm_amd import head
    return head


def test_library_exports_what_the_header_declares(hd):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(mq_[a-z0-9_]+)\s*\(", src)))
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T " in l) == declared == sorted(hd.EXPORTED)


def _quantize(hd, x=A, M=3, K=200, xs=200, c=A, cs=256, s=A, ss=2):
    return hd.lib.mq_quantize8(x, M, K, xs, c, cs, s, ss, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(x=A + 1), BAD), (dict(M=-1), BAD), (dict(K=0), BAD), (dict(xs=199), BAD),
    (dict(c=None), BAD), (dict(c=A + 8), BAD), (dict(cs=240), BAD), (dict(cs=264), BAD), (dict(s=None), BAD),
    (dict(ss=1), BAD), (dict(K=(1 << 20) + 1, xs=1 << 21, cs=1 << 21, ss=1 << 14), UNS), (dict(M=1 << 31), UNS),
    (dict(M=1 << 23, K=1 << 20, xs=1 << 20, cs=1 << 20, ss=1 << 13), UNS),
])
def test_quantize_refusals(hd, kw, code):
    assert _quantize(hd, **kw) == code


def test_nothing_is_enqueued_for_no_rows(hd):
    assert _quantize(hd, M=0) == 0
    assert _linear(hd, M=0) == 0
    assert _sample(hd, rows=0) == 0


def _w8(hd, **kw):
    return hd._W8(**(dict(codes=A, scales=A, N=100, K=200) | kw))


@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), BAD), (dict(codes=A + 8), BAD), (dict(scales=None), BAD), (dict(scales=A + 2), BAD),
    (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=(1 << 20) + 1), UNS), (dict(N=(1 << 24) + 1), UNS),
    (dict(N=1 << 21, K=1 << 20), UNS),
])
def test_weights_refusals(hd, kw, code):
    w = _w8(hd, **kw)
    assert hd.lib.mq_pack8(A, 1 << 21, ctypes.byref(w), None) == code
    assert _linear(hd, w=kw, cs=1 << 21, ss=1 << 14, ys=1 << 25) == code


def test_pack_refusals(hd):
    w = _w8(hd)
    for x, stride in ((None, 200), (A + 1, 200), (A, 199)):
        assert hd.lib.mq_pack8(x, stride, ctypes.byref(w), None) == BAD
    assert hd.lib.mq_pack8(A, 200, None, None) == BAD
    n = ctypes.c_size_t()
    assert hd.lib.mq_pack8_bytes(100, 200, None, ctypes.byref(n)) == BAD
    assert hd.lib.mq_pack8_bytes(0, 200, ctypes.byref(n), ctypes.byref(n)) == BAD
    c = ctypes.c_size_t()
    assert hd.lib.mq_pack8_bytes(100, 700, ctypes.byref(c), ctypes.byref(n)) == 0
    assert (c.value, n.value) == (7 * 6 * 2048, 7 * 2 * 64)


def _linear(hd, c=A, cs=256, s=A, ss=2, M=3, w={}, y=A, ys=100, ws=A, nws=1 << 40):
    return hd.lib.mq_linear8(c, cs, s, ss, M, ctypes.byref(_w8(hd, **w)), y, ys, ws, nws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), BAD), (dict(c=A + 8), BAD), (dict(cs=240), BAD), (dict(cs=260), BAD), (dict(s=None), BAD),
    (dict(ss=1), BAD), (dict(M=-1), BAD), (dict(y=None), BAD), (dict(y=A + 1), BAD), (dict(ys=99), BAD),
    (dict(M=100, w=dict(K=40960), cs=40960, ss=320, nws=16), BAD), (dict(M=100, w=dict(K=40960), cs=40960, ss=320, ws=None), BAD),
    (dict(M=100, w=dict(K=40960), cs=40960, ss=320, ws=A + 8), BAD), (dict(M=1 << 24), UNS), (dict(cs=(1 << 22) + 16), UNS),
    (dict(ss=(1 << 22) + 1), UNS),
    (dict(M=(1 << 24) - 1, w=dict(N=1 << 24, K=128), cs=128, ss=1, ys=1 << 24), UNS),
])
def test_linear_refusals(hd, kw, code):
    assert _linear(hd, **kw) == code


def test_linear_workspace(hd):
    n = ctypes.c_size_t(7)

    def size(M, **kw):
        st = hd.lib.mq_linear8_workspace(M, ctypes.byref(_w8(hd, **kw)), ctypes.byref(n))
        return st, n.value
    assert size(16, N=4096, K=4096) == (0, 0)                     # few tokens: none
    st, b = size(100, N=64, K=40960)                              # few outputs of long sums: split along K
    assert st == 0 and b > 0 and b % (100 * 64 * 4) == 0
    assert hd.lib.mq_linear8_workspace(16, ctypes.byref(_w8(hd)), None) == BAD
    assert hd.lib.mq_linear8_workspace(16, None, ctypes.byref(n)) == BAD
    assert size(-1)[0] == BAD


def _sample(hd, ws=A, nws=1 << 40, **kw):
    a = hd._SampleArgs(**(dict(logits=A, rows=3, vocab=100, stride=100, u=A, token=A) | kw))
    return hd.lib.mq_sample(ctypes.byref(a), ws, nws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), BAD), (dict(logits=A + 1), BAD), (dict(logits=A + 2, logits_fp32=1), BAD), (dict(rows=-1), BAD),
    (dict(vocab=0), BAD), (dict(stride=99), BAD), (dict(u=None), BAD), (dict(token=None), BAD), (dict(u=A + 2), BAD),
    (dict(token=A + 2), BAD), (dict(logprob=A + 2), BAD), (dict(temperature=A + 2), BAD), (dict(top_k=A + 1), BAD),
    (dict(top_p=A + 2), BAD), (dict(min_p=A + 2), BAD), (dict(logits_fp32=2), BAD), (dict(rows=65536), UNS),
    (dict(vocab=(1 << 22) + 1, stride=1 << 23), UNS),
])
def test_sample_refusals(hd, kw, code):
    assert _sample(hd, **kw) == code


def test_sample_refuses_missing_arguments(hd):
    n = ctypes.c_size_t()
    assert hd.lib.mq_sample(None, A, 1 << 30, None) == BAD
    assert hd.lib.mq_sample_workspace(None, ctypes.byref(n)) == BAD
    a = hd._SampleArgs(rows=3, vocab=100)
    assert hd.lib.mq_sample_workspace(ctypes.byref(a), None) == BAD
    assert hd.lib.mq_sample_workspace(ctypes.byref(a), ctypes.byref(n)) == 0


def test_sample_arguments_are_packed_as_the_structure_lies(hd):
    a = hd._SampleArgs.from_buffer_copy(hd._sample_args(*range(1, 13)))
    assert [getattr(a, n) for n, _ in hd._SampleArgs._fields_] == list(range(1, 13))


# ------------------------------------------------------------- norm to 8 bits
def _norm(bk, scales=A, ss=1, **kw):
    f = dict(y=A, r=A, w_pre=A, r_out=A, h_out=A, tokens=2, width=100, y_stride=100, r_stride=100, r_out_stride=100,
             h_stride=128, alpha=1.0, beta=1.0, eps=1e-6) | kw
    return bk.lib.mq_norm_residual_q8(ctypes.byref(bk._NormArgs(**f)), scales, ss, None)


@pytest.mark.parametrize("kw", [
    dict(w_pre=None), dict(h_out=None), dict(h_out=A + 8), dict(h_stride=112), dict(h_stride=136), dict(scales=None),
    dict(ss=0), dict(r=None), dict(r_out=None), dict(tokens=-1), dict(width=0), dict(y_stride=99), dict(eps=-1.0),
    dict(alpha=float("nan")), dict(residual_fp32=2), dict(weight_offset=float("inf")),
])
def test_norm_refusals(bk, kw):  # noqa: F811
    assert _norm(bk, **kw) == BAD


def test_norm_refuses_rows_that_are_too_wide(bk):  # noqa: F811
    w = 65537
    assert _norm(bk, width=w, y_stride=w, r_stride=w, r_out_stride=w, h_stride=513 * 128, ss=513) == UNS
    assert bk.lib.mq_norm_residual_q8(None, A, 1, None) == BAD
