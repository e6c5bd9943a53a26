"""What the head's binding refuses, without a GPU: tensors that say they are on one stand in for those that are (nothing
here reaches a launch)."""
import pytest
import torch

from tests.test_block_abi_cpu import bk  # noqa: F401  (the fixtures)
from tests.test_block_binding_cpu import OnGpu, gpu
from tests.test_head_abi_cpu import hd  # noqa: F401

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class OnOther(OnGpu):
    """On GPU 1."""

    def get_device(self):
        return 1


def bytes_(shape, dt, kind=OnGpu):
    return torch.zeros(shape, dtype=torch.uint8).view(dt).as_subclass(kind)


def layer(hd, N=100, K=200, kind=OnGpu):  # noqa: F811
    return hd.Packed8(gpu(7 * 2 * 2048, torch.uint8, kind), gpu(7 * 64, torch.uint8, kind), N, K)


def test_rows_of_other_shapes_and_types_are_refused(hd, monkeypatch):  # noqa: F811
    monkeypatch.setattr(hd, "_current_device", lambda: 0)
    x = gpu((3, 200))
    with pytest.raises(TypeError):
        hd.mq_quantize8(torch.zeros((3, 200), dtype=torch.float16))
    with pytest.raises(TypeError):
        hd.mq_quantize8(gpu((3, 200), torch.float32))
    with pytest.raises(ValueError):
        hd.mq_quantize8(gpu((3, 200, 2)))
    for c, s in (((3, 200), (3, 2)), ((2, 256), (3, 2)), ((3, 256), (3, 1))):
        with pytest.raises(ValueError):
            hd.mq_quantize8(x, bytes_(c, F8), bytes_(s, E8))
    with pytest.raises(TypeError):
        hd.mq_quantize8(x, gpu((3, 256), torch.uint8), bytes_((3, 2), E8))
    with pytest.raises(TypeError):
        hd.mq_quantize8(x, bytes_((3, 256), F8), gpu((3, 2), torch.float32))


def test_layers_are_checked(hd):  # noqa: F811
    c, s = gpu(7 * 2 * 2048, torch.uint8), gpu(7 * 64, torch.uint8)
    for args, err in (((c[:-1], s, 100, 200), ValueError), ((c, s[:-1], 100, 200), ValueError),
                      ((c.to(torch.int8), s, 100, 200), TypeError), ((c, s, 113, 200), ValueError),
                      ((c, gpu(7 * 64, torch.uint8, OnOther), 100, 200), ValueError), ((c, s, 0, 200), hd.MQError)):
        with pytest.raises(err):
            hd.Packed8(*args)
    assert hd.Packed8(c, s, 100, 200).device_bytes == 7 * (2 * 2048 + 64)


def test_linear_refuses(hd, monkeypatch):  # noqa: F811
    monkeypatch.setattr(hd, "_current_device", lambda: 0)
    c, s, p = bytes_((3, 256), F8), bytes_((3, 2), E8), layer(hd)
    with pytest.raises(ValueError):
        hd.mq_linear8(c, s, layer(hd, kind=OnOther))
    with pytest.raises(ValueError):
        hd.mq_linear8(bytes_((3, 384), F8), bytes_((3, 3), E8), p)
    with pytest.raises(ValueError):
        hd.mq_linear8(c, bytes_((2, 2), E8), p)
    with pytest.raises(TypeError):
        hd.mq_linear8(gpu((3, 256)), s, p)
    with pytest.raises(ValueError):
        hd.mq_linear8(c, s, p, out=gpu((3, 99)))
    with pytest.raises(TypeError):
        hd.mq_linear8(c, s, p, out=gpu((3, 100), torch.float32))
    with pytest.raises(TypeError):
        hd.mq_linear8(c, s, p, out=gpu((3, 100)), workspace=gpu(64, torch.int32))


def test_sample_refuses(hd, monkeypatch):  # noqa: F811
    monkeypatch.setattr(hd, "_current_device", lambda: 0)
    l, u = gpu((3, 50)), gpu(3, torch.float32)
    out = dict(token_out=gpu(3, torch.int32), logprob_out=gpu(3, torch.float32))
    with pytest.raises(TypeError):
        hd.mq_sample(torch.zeros((3, 50)), u, **out)
    with pytest.raises(TypeError):
        hd.mq_sample(gpu((3, 50), torch.int32), u, **out)
    with pytest.raises(ValueError):
        hd.mq_sample(gpu(50), u, **out)
    with pytest.raises(TypeError):
        hd.mq_sample(l, None, **out)
    with pytest.raises(ValueError):
        hd.mq_sample(l, gpu(2, torch.float32), **out)
    for name, t in (("temperature", gpu(3)), ("top_k", gpu(3, torch.int64)), ("top_p", gpu(3, torch.float64)),
                    ("min_p", gpu(3)), ("token_out", gpu(3, torch.int64)), ("logprob_out", gpu(3))):
        with pytest.raises(TypeError, match=name):
            hd.mq_sample(l, u, **(out | {name: t}))
    with pytest.raises(ValueError, match="top_k"):
        hd.mq_sample(l, u, top_k=gpu((3, 1), torch.int32), **out)
    with pytest.raises(TypeError, match="workspace"):
        hd.mq_sample(l, u, workspace=gpu(64, torch.float32), **out)


def test_norm_to_8_bits_refuses(bk, monkeypatch):  # noqa: F811
    monkeypatch.setattr(bk, "_current_device", lambda: 0)
    y, r, w = gpu((3, 200)), gpu((3, 200)), gpu(200)
    with pytest.raises(TypeError):
        bk.mq_norm_residual_q8(y, r, None, r_out=r)
    with pytest.raises(ValueError):
        bk.mq_norm_residual_q8(y, r, w, r_out=r, codes_out=bytes_((3, 200), F8), scales_out=bytes_((3, 2), E8))
    with pytest.raises(TypeError):
        bk.mq_norm_residual_q8(y, r, w, r_out=r, codes_out=bytes_((3, 256), F8), scales_out=gpu((3, 2), torch.uint8))
    with pytest.raises(ValueError):
        bk.mq_norm_residual_q8(gpu((2, 200)), r, w, r_out=r, codes_out=bytes_((3, 256), F8), scales_out=bytes_((3, 2), E8))
