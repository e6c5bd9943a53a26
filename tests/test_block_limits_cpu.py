"""Bounds of the block operators that no launch can take (2^32 threads), without a GPU: refused before any HIP call."""
import ctypes

import pytest

from tests.test_block_abi_cpu import UNS, _append, _batch, _cache, bk  # noqa: F401  (bk: the fixture)


@pytest.mark.parametrize("seqs,max_new,kv_heads,queries", [
    (256, 131072, 32, False),            # 2049 blocks a sequence, 32 heads
    (65535, 1, 257, False),              # a block a sequence
    (512, 131072, 1, True),              # 32768 workgroups of queries a sequence
])
def test_append_refuses_what_no_launch_takes(bk, seqs, max_new, kv_heads, queries):
    w = 64 * kv_heads
    q = dict(rope={}, q=1 << 20, heads=1, qs=64, qo=1 << 20, qos=64) if queries else {}
    assert _append(bk, cache=dict(kv_heads=kv_heads), batch=dict(seqs=seqs, tokens=1 << 28, max_new=max_new), ks=w, vs=w,
                   **q) == UNS


@pytest.mark.parametrize("ok,over,D,heads", [
    # many rows of 128: workgroups of 512 threads
    (dict(seqs=4095, tokens=1 << 28, max_new=65536), dict(seqs=4096, tokens=1 << 28, max_new=65536), 128, (8, 8)),
    # of 64: of 256
    (dict(seqs=4095, tokens=1 << 28, max_new=65536), dict(seqs=4096, tokens=1 << 28, max_new=65536), 64, (8, 8)),
    # few rows
    (dict(seqs=65535, tokens=65535), dict(seqs=65535, tokens=65535), 64, (256, 257)),
    # the join of a split cache: a workgroup a row; 16 rows in few splits
    (dict(seqs=1, tokens=(1 << 24) - 1, max_len=1 << 20), dict(seqs=1, tokens=1 << 24, max_len=1 << 20), 64, (1, 1)),
    (dict(seqs=1, tokens=(1 << 28) - 16, max_len=1024), dict(seqs=1, tokens=1 << 28, max_len=1024), 64, (1, 1)),
])
def test_attention_refuses_what_no_launch_takes(bk, ok, over, D, heads):
    n = ctypes.c_size_t()

    def size(batch, hk):
        c = _cache(bk, head_dim=D, kv_heads=hk)
        return bk.lib.mq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(_batch(bk, **batch)), hk, ctypes.byref(n))
    assert size(ok, heads[0]) == 0
    assert size(over, heads[1]) == UNS
