"""C ABI of the block operators, without a GPU: the library exports exactly
what include/mosaicq_block.h declares and refuses bad arguments before any
HIP call."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_gemm_amd", "libmosaicq_block.so")
HEADER = os.path.join(ROOT, "include", "mosaicq_block.h")
A = 1 << 20                     # an aligned address that validation never reads
BAD, UNS = -1, -2


@pytest.fixture(scope="module")
def bk():
    assert os.path.exists(LIB), "libmosaicq_block.so is not built (python -m bit_gemm_amd.build)"
    from bit_gemm_amd import block
    return block


def test_library_exports_what_the_header_declares(bk):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(mq_[a-z0-9_]+)\s*\(", src)))
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T " in l) == declared == sorted(bk.EXPORTED)


def _table(bk, positions=16, table=A, **kw):
    f = dict(rot_dim=64, scaling=0, theta=1e4, factor=1.0, original=8192.0, turns_fast=32.0, turns_slow=1.0) | kw
    return bk.lib.mq_rope_table(ctypes.byref(bk._RopeSpec(**f)), positions, table, None)


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), BAD), (dict(table=A + 4), BAD), (dict(positions=0), BAD), (dict(rot_dim=0), BAD),
    (dict(rot_dim=63), BAD), (dict(rot_dim=1026), BAD), (dict(scaling=4), BAD), (dict(theta=1.0), BAD),
    (dict(theta=float("nan")), BAD), (dict(scaling=1, factor=0.5), BAD), (dict(scaling=2, factor=float("inf")), BAD),
    (dict(scaling=3, original=0.0), BAD), (dict(scaling=3, turns_fast=1.0), BAD), (dict(scaling=3, turns_slow=0.0), BAD),
    (dict(positions=(1 << 31) // 64), UNS),
])
def test_rope_table_refusals(bk, kw, code):
    assert _table(bk, **kw) == code


def _plan(bk, **kw):
    return bk._RopePlan(**(dict(table=A, positions=100, rot_dim=64, layout=0) | kw))


def _rope(bk, x=A, tokens=3, heads=4, dim=64, xt=256, xh=64, pos=A, inverse=0, y=A, yt=256, yh=64, rope=True, **kw):
    plan = _plan(bk, **kw)
    return bk.lib.mq_rope(x, tokens, heads, dim, xt, xh, pos, ctypes.byref(plan) if rope else None, inverse, y, yt, yh,
                          None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(pos=None), BAD), (dict(rope=False), BAD), (dict(tokens=-1), BAD),
    (dict(heads=0), BAD), (dict(dim=1), BAD), (dict(x=A + 1), BAD), (dict(pos=A + 2), BAD), (dict(inverse=2), BAD),
    (dict(xt=-1), BAD), (dict(yh=63), BAD), (dict(yt=63), BAD), (dict(table=None), BAD), (dict(table=A + 4), BAD),
    (dict(positions=0), BAD), (dict(rot_dim=66), BAD), (dict(rot_dim=7), BAD), (dict(layout=2), BAD),
    (dict(tokens=1 << 31), UNS), (dict(heads=1 << 25), UNS),
])
def test_rope_refusals(bk, kw, code):
    assert _rope(bk, **kw) == code


def test_rope_of_no_tokens_does_nothing(bk):
    assert _rope(bk, tokens=0) == 0


def _cache(bk, **kw):
    return bk._Cache(**(dict(k_codes=A, v_codes=A, k_scale=A, v_scale=A, k_tail=A, v_tail=A, num_blocks=8, num_slots=2,
                             kv_heads=2, head_dim=64, format=0) | kw))


def _batch(bk, **kw):
    return bk._Batch(**(dict(cu_q=A, kv_len=A, block_table=A, slots=None, seqs=2, tokens=2, table_width=4, max_new=1,
                             max_len=100) | kw))


CACHE_BAD = [(dict(k_codes=None), BAD), (dict(v_codes=A + 8), BAD), (dict(k_scale=None), BAD), (dict(v_scale=A + 2), BAD),
             (dict(k_tail=None), BAD), (dict(v_tail=A + 4), BAD), (dict(num_blocks=0), BAD), (dict(num_slots=0), BAD),
             (dict(kv_heads=0), BAD), (dict(kv_heads=1025), BAD), (dict(format=2), BAD), (dict(head_dim=96), UNS),
             (dict(head_dim=256), UNS)]
BATCH_BAD = [(dict(cu_q=None), BAD), (dict(kv_len=A + 1), BAD), (dict(block_table=None), BAD), (dict(slots=A + 2), BAD),
             (dict(seqs=-1), BAD), (dict(seqs=65536), BAD), (dict(tokens=-1), BAD), (dict(table_width=0), BAD),
             (dict(max_new=0), BAD), (dict(max_len=0), BAD), (dict(tokens=1 << 31), UNS), (dict(max_len=1 << 31), UNS),
             (dict(table_width=1 << 31), UNS)]


def _append(bk, cache={}, batch={}, q=None, heads=0, qs=0, k=A, ks=128, v=A, vs=128, rope=None, qo=None, qos=0):
    c, b = _cache(bk, **cache), _batch(bk, **batch)
    r = None if rope is None else ctypes.byref(_plan(bk, **rope))
    return bk.lib.mq_kv_append(ctypes.byref(c), ctypes.byref(b), q, heads, qs, k, ks, v, vs, r, qo, qos, None)


def _attend(bk, cache={}, batch={}, q=A, heads=8, qs=512, causal=1, scale=0.125, o=A, os=512, ws=A, nws=1 << 30):
    c, b = _cache(bk, **cache), _batch(bk, **batch)
    return bk.lib.mq_kv_attention(ctypes.byref(c), ctypes.byref(b), q, heads, qs, causal, scale, o, os, ws, nws, None)


@pytest.mark.parametrize("kw,code", CACHE_BAD)
def test_cache_refusals(bk, kw, code):
    assert _append(bk, cache=kw) == code
    assert _attend(bk, cache=kw) == code


@pytest.mark.parametrize("kw,code", BATCH_BAD)
def test_batch_refusals(bk, kw, code):
    assert _append(bk, batch=kw) == code
    assert _attend(bk, batch=kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=A + 1), BAD), (dict(ks=127), BAD), (dict(vs=0), BAD),
    (dict(rope=dict(rot_dim=66)), BAD), (dict(rope=dict(table=None)), BAD),
    (dict(rope={}, q=A, heads=4, qs=256, qo=None, qos=256), BAD), (dict(rope={}, q=A, heads=0, qs=256, qo=A, qos=256), BAD),
    (dict(rope={}, q=A, heads=4, qs=255, qo=A, qos=256), BAD), (dict(rope={}, q=A, heads=4, qs=256, qo=A, qos=255), BAD),
    (dict(batch=dict(seqs=65535, tokens=(1 << 31) - 1, max_new=(1 << 31) - 1)), UNS),
])
def test_append_refusals(bk, kw, code):
    assert _append(bk, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(q=A + 8), BAD), (dict(qs=516), BAD), (dict(qs=504), BAD),
    (dict(o=A + 4), BAD), (dict(os=514), BAD), (dict(os=508), BAD), (dict(heads=0), BAD), (dict(heads=7), BAD),
    (dict(heads=130, qs=130 * 64, os=130 * 64), UNS), (dict(causal=2), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD),
    (dict(batch=dict(max_len=100000), nws=64), BAD), (dict(batch=dict(max_len=100000), ws=None), BAD),
    (dict(batch=dict(max_len=100000), ws=A + 8), BAD),
    (dict(batch=dict(seqs=65535, tokens=(1 << 31) - 1, max_new=(1 << 31) - 1)), UNS),
])
def test_attention_refusals(bk, kw, code):
    assert _attend(bk, **kw) == code


def test_workspace_sizes(bk):
    n = ctypes.c_size_t(7)
    c = _cache(bk)

    def size(**kw):
        st = bk.lib.mq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(_batch(bk, **kw)), 8, ctypes.byref(n))
        return (st, n.value)
    assert size() == (0, 0)                                      # a short cache is not split
    st, a = size(max_len=1 << 20)
    assert st == 0 and a > 0
    assert bk.lib.mq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(_batch(bk)), 8, None) == BAD
    assert bk.lib.mq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(_batch(bk)), 7, ctypes.byref(n)) == BAD
    # no rows, nothing to do, no pointers read
    assert _attend(bk, batch=dict(seqs=0)) == 0 and _append(bk, batch=dict(tokens=0)) == 0


def _norm(bk, **kw):
    f = dict(y=A, r=A, gate=None, w_post=None, w_pre=A, r_out=A, h_out=A, tokens=2, width=64, y_stride=64, r_stride=64,
             gate_stride=0, r_out_stride=64, h_stride=64, alpha=1.0, beta=1.0, eps=1e-6, weight_offset=0.0,
             residual_fp32=0) | kw
    return bk.lib.mq_norm_residual(ctypes.byref(bk._NormArgs(**f)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(r=None), BAD), (dict(r=A + 1), BAD), (dict(r=A + 2, residual_fp32=1), BAD), (dict(y=None, w_pre=None), BAD),
    (dict(r_out=None), BAD), (dict(h_out=None), BAD), (dict(tokens=-1), BAD), (dict(width=0), BAD),
    (dict(y_stride=63), BAD), (dict(r_stride=0), BAD), (dict(r_out_stride=1), BAD), (dict(h_stride=8), BAD),
    (dict(gate=A, gate_stride=63), BAD), (dict(gate=A + 1), BAD), (dict(w_post=A + 1), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(alpha=float("inf")), BAD), (dict(weight_offset=float("nan")), BAD),
    (dict(residual_fp32=2), BAD), (dict(tokens=1 << 31), UNS),
    (dict(width=65537, y_stride=65537, r_stride=65537, r_out_stride=65537, h_stride=65537), UNS),
])
def test_norm_refusals(bk, kw, code):
    assert _norm(bk, **kw) == code


def test_norm_of_no_tokens_does_nothing(bk):
    assert _norm(bk, tokens=0) == 0


def test_binding_checks_arguments(bk):
    import torch
    host = torch.zeros((2, 4, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        bk.mq_rope(host, None, None)
    with pytest.raises(TypeError):
        bk.mq_norm_residual(None, host[0], None)
    with pytest.raises(TypeError):
        bk.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1)), 1, 1)
    with pytest.raises(TypeError):
        bk.KVCache(*[host] * 6)
    with pytest.raises(ValueError):
        bk.Rope(64, 10, layout="other")


def test_norm_arguments_are_packed_as_the_structure_lies(bk):
    v = (1, 2, 3, 0, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 0.5, 0.25, 2.0, 4.0, True)
    a = bk._NormArgs(*v)
    assert bk._norm_args(*v) == bytes(a)
