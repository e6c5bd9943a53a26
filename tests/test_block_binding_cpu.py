"""What the block operators' binding refuses, and what it hands to the library, without a GPU: tensors that say they are on
one stand in for those that are (nothing here reaches a launch)."""
import ctypes

import pytest
import torch

from tests.test_block_abi_cpu import bk  # noqa: F401  (the fixture)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def gpu(shape, dtype=torch.float16, kind=OnGpu):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def cache_of(bk, kind=OnGpu, **other):
    """A cache of 4 blocks, 2 slots, 2 kv heads of 64; other: tensors of another kind."""
    shapes = {"k_codes": ((4, 2, 64, 64), torch.int8), "v_codes": ((4, 2, 64, 64), torch.int8),
              "k_scale": ((4, 2), torch.float32), "v_scale": ((4, 2), torch.float32),
              "k_tail": ((2, 2, 64, 64), torch.float16), "v_tail": ((2, 2, 64, 64), torch.float16)}
    return bk.KVCache(*[gpu(*shapes[n], kind=other.get(n, kind)) for n in shapes])


def batch_of(bk, kind=OnGpu, **other):
    shapes = {"cu_q": (3,), "kv_len": (2,), "block_table": (2, 4), "slots": (2,)}
    t = {n: gpu(shapes[n], torch.int32, other.get(n, kind)) for n in shapes}
    return bk.KVBatch(t["cu_q"], t["kv_len"], t["block_table"], 1, 100, slots=t["slots"])


class NoPlan:
    """Stands for a rope plan where the call is refused before it is read."""
    _ref = 0


def test_append_refuses_an_output_that_it_would_not_write(bk):
    q, kv, out = gpu((2, 4, 64)), gpu((2, 2, 64)), gpu((2, 4, 64))
    for args, kw in (((q, kv, kv), {}), ((None, kv, kv), {}), ((None, kv, kv), dict(rope=NoPlan()))):
        with pytest.raises(ValueError, match="q_out"):
            bk.mq_kv_append(*args, cache_of(bk), batch_of(bk), q_out=out, **kw)


def test_calls_of_one_batch_do_not_share_their_token_count(bk):
    """Two threads may run calls of one batch with different numbers of tokens: each call's structure is its own."""
    b = batch_of(bk)

    def tokens(args):
        p = args if isinstance(args, bytes) else ctypes.string_at(args, ctypes.sizeof(bk._Batch))
        return bk._Batch.from_buffer_copy(p).tokens
    two, three = b._with(2), b._with(3)
    assert (tokens(two), tokens(three)) == (2, 3)


def test_batch_arguments_are_packed_as_the_structure_lies(bk):
    b = batch_of(bk)
    want = bk._Batch(b.cu_q.data_ptr(), b.kv_len.data_ptr(), b.block_table.data_ptr(), b.slots.data_ptr(), 2, 7, 4, 1, 100)
    assert b._with(7) == bytes(want)
    none = bk.KVBatch(b.cu_q, b.kv_len, b.block_table, 1, 100)
    assert bk._Batch.from_buffer_copy(none._with(7)).slots is None
