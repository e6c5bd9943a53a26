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


class Elsewhere(OnGpu):
    """Says it is on GPU 1."""

    def get_device(self):
        return 1


def test_tensors_of_different_devices_are_refused(bk, monkeypatch):
    monkeypatch.setattr(bk, "_current_device", lambda: 0)
    for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
        with pytest.raises((TypeError, ValueError), match="device|GPU"):
            cache_of(bk, **{n: Elsewhere})
    for n in ("cu_q", "kv_len", "block_table", "slots"):
        with pytest.raises((TypeError, ValueError), match="device|GPU"):
            batch_of(bk, **{n: Elsewhere})
    c, b = cache_of(bk), batch_of(bk)
    q, kv = gpu((2, 4, 64)), gpu((2, 2, 64))
    far = [gpu((2, 4, 64), kind=Elsewhere), gpu((2, 2, 64), kind=Elsewhere)]
    plan = bk.Rope.__new__(bk.Rope)
    plan.device, plan._ref, plan.rot_dim = 0, 0, 64
    calls = [
        lambda: bk.mq_kv_append(None, far[1], kv, c, b), lambda: bk.mq_kv_append(None, kv, far[1], c, b),
        lambda: bk.mq_kv_append(far[0], kv, kv, c, b, rope=plan),
        lambda: bk.mq_kv_append(q, kv, kv, c, b, rope=plan, q_out=far[0]),
        lambda: bk.mq_kv_append(None, kv, kv, cache_of(bk, Elsewhere), b),
        lambda: bk.mq_kv_append(None, kv, kv, c, batch_of(bk, Elsewhere)),
        lambda: bk.mq_kv_attention(far[0], c, b), lambda: bk.mq_kv_attention(q, c, b, out=far[0]),
        lambda: bk.mq_kv_attention(q, c, batch_of(bk, Elsewhere)),
        lambda: bk.mq_kv_attention(q, cache_of(bk, Elsewhere), b),
        lambda: bk.mq_rope(far[0], plan, gpu((2,), torch.int32)),
        lambda: bk.mq_rope(q, plan, gpu((2,), torch.int32, Elsewhere)),
        lambda: bk.mq_rope(q, plan, gpu((2,), torch.int32), out=far[0]),
    ]
    r, w, y = gpu((2, 64)), gpu((64,)), gpu((2, 64))
    for name in ("y", "w_pre", "w_post", "gate", "r_out", "h_out"):
        a = dict(y=y, w_pre=w, w_post=w, gate=w, r_out=gpu((2, 64)), h_out=gpu((2, 64)))
        a[name] = gpu(a[name].shape, kind=Elsewhere)
        calls.append(lambda a=a: bk.mq_norm_residual(a.pop("y"), r, a.pop("w_pre"), **a))
    plan.device = 1
    calls.append(lambda: bk.mq_kv_append(q, kv, kv, c, b, rope=plan))
    for i, call in enumerate(calls):
        plan.device = 1 if i == len(calls) - 1 else 0
        with pytest.raises((TypeError, ValueError), match="device|GPU"):
            call()


def test_calls_run_on_their_tensors_device(bk, monkeypatch):
    """Where the current device is another one, it is the tensors' for the call alone."""
    seen, now = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, now[0]))
                return 0
            return call
    monkeypatch.setattr(bk, "lib", Library())
    monkeypatch.setattr(bk, "_current_device", lambda: now[0])
    monkeypatch.setattr(bk, "_current_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for kind, device in ((OnGpu, 0), (Elsewhere, 1)):
        c, b = cache_of(bk, kind), batch_of(bk, kind)
        q, kv = gpu((2, 4, 64), kind=kind), gpu((2, 2, 64), kind=kind)
        r, w = gpu((2, 64), kind=kind), gpu((64,), kind=kind)
        plan = bk.Rope.__new__(bk.Rope)
        plan.device, plan._ref, plan.rot_dim = device, 0, 64
        del seen[:]
        bk.mq_kv_append(q, kv, kv, c, b, rope=plan, q_out=q)
        bk.mq_kv_attention(q, c, b, out=q)
        bk.mq_rope(q, plan, gpu((2,), torch.int32, kind), out=q)
        bk.mq_norm_residual(r, r, w, r_out=r, h_out=r)
        assert [d for name, d in seen if name != "mq_kv_attention_workspace"] == [device] * 4
        assert now[0] == 0
