"""Calls of the linears' binding on a stream that is not the current one: what they make comes from that stream's memory,
and the values are those of a call on the current one."""
import numpy as np
import pytest

from tests.gpu_util import require_gpu, to_dev

pytestmark = pytest.mark.gpu


def freed(nbytes):
    """The addresses of a block of this size that the current stream's pool has just got back."""
    import torch
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    return range(at, at + nbytes)


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream_are_not_the_current_ones_memory(raw):
    import torch
    mq = require_gpu()
    N, K, M = 256, 512, 2
    W = to_dev((np.random.default_rng(1).standard_normal((N, K)) * 0.02).astype(np.float16))
    X = to_dev(np.random.default_rng(2).standard_normal((M, K)).astype(np.float16))
    p, plain = mq.mq_pack(W, 128, 0.01), mq.mq_pack(W, 128, 0.0)
    amax = X.float().abs().amax(0)
    codes, meta = mq.mq_quantize_activations(X, 128)
    e = mq.mq_smooth_weights(W, amax)[1]
    strided = torch.stack([amax, amax], 1)[:, 0]
    y = M * N * 2
    calls = {
        "linear": (lambda s: [mq.mq_linear(X, p, stream=s)], y),
        "group": (lambda s: mq.mq_linear_group([X, X], [p, p], stream=s), y),
        "quantize": (lambda s: list(mq.mq_quantize_activations(X, 128, stream=s)), M * K),
        "linear_a4": (lambda s: [mq.mq_linear_a4(codes, meta, plain, stream=s)], y),
        "decode_a4": (lambda s: [mq.mq_decode_a4(X, plain, stream=s)], y),
        "smooth_activations": (lambda s: [mq.mq_smooth_activations(X, e, stream=s)], M * K * 2),
        "smooth_weights": (lambda s: list(mq.mq_smooth_weights(W, amax, stream=s)), N * K * 2),
        "smooth_weights of a strided maximum": (lambda s: list(mq.mq_smooth_weights(W, strided, stream=s)), K * 4),
        "export_canonical": (lambda s: list(mq.mq_export_canonical(p, stream=s).values()), N * K // 2),
        "export_tiled": (lambda s: list(mq.mq_export_tiled(p, stream=s).values()), N * K // 2),
    }
    side = torch.cuda.Stream()
    for name, (call, nbytes) in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        block = freed(nbytes)
        got = call(side.cuda_stream if raw else side)
        side.synchronize()
        assert all(t.data_ptr() not in block for t in got), name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_any_object_with_a_stream_handle_is_taken():
    """A stream of another library, which is known by its cuda_stream alone."""
    import torch
    mq = require_gpu()

    class Handle:
        def __init__(self, stream):
            self.stream, self.cuda_stream = stream, stream.cuda_stream
    W = to_dev((np.random.default_rng(3).standard_normal((64, 128)) * 0.02).astype(np.float16))
    X = to_dev(np.random.default_rng(4).standard_normal((3, 128)).astype(np.float16))
    p = mq.mq_pack(W, 128, 0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mq.mq_linear(X, p, stream=Handle(side))
    side.synchronize()
    assert torch.equal(y, mq.mq_linear(X, p))
