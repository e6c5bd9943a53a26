"""Python binding of include/mosaicq_head.h (ctypes): the way out of a model.

    codes, scales = mq_quantize8(x)                         # fp16 rows as 8-bit rows
    r, codes, scales = block.mq_norm_residual_q8(y, r, w)   # or straight from the last norm
    layer = mq_pack8(W)                                     # weights in 8 bits
    logits = mq_linear8(codes, scales, layer)
    token, logprob = mq_sample(logits, u, temperature=t, top_k=k, top_p=p)

8-bit rows are codes float8_e4m3fn [rows, 128 n] and scales float8_e8m0fnu
[rows, n], n = ceil(width / 128), a power of two for each block of 128.

Argument marshalling only: every step runs in the HIP library, on the given
stream (the current one by default) of its tensors' device, without
synchronising. What a call makes (outputs, workspace) comes from that stream's
memory pool; the caller orders the streams, and keeps what a call reads until
it has run. Importing this module fails loudly when the library is not built --
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from .block import _apart, _current_device, _device, _E4M3, _E8M0, _F16, _matrix, _rows8, _rows8_out, _stream
from .mosaicq import MQError, _check, _new, _other

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmosaicq_head.so")

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_size = ctypes.c_size_t


class _W8(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("N", _i64), ("K", _i64)]


class _SampleArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("rows", _i64), ("vocab", _i64), ("stride", _i64)] + [
        (n, _vp) for n in ("temperature", "top_k", "top_p", "min_p", "u", "token", "logprob")] + [("logits_fp32", _i32)]


# the same fields in their order, packed at once
_sample_args = struct.Struct("@P3q7Pi4x").pack

EXPORTED = ("mq_quantize8", "mq_pack8_bytes", "mq_pack8", "mq_linear8", "mq_linear8_workspace", "mq_sample",
            "mq_sample_workspace")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built (run `python -m bit_gemm_amd.build`)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.mq_quantize8.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]
    lib.mq_pack8_bytes.argtypes = [_i64, _i64, _vp, _vp]
    lib.mq_pack8.argtypes = [_vp, _i64, _vp, _vp]
    lib.mq_linear8.argtypes = [_vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _size, _vp]
    lib.mq_linear8_workspace.argtypes = [_i64, _vp, _vp]
    lib.mq_sample.argtypes = [_vp, _vp, _size, _vp]
    lib.mq_sample_workspace.argtypes = [_vp, _vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def _half_matrix(t, name: str):
    """Device, rows, width and row stride of a float16 [rows, width] tensor with dense rows."""
    device = _device(t, name, _F16)
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be [rows, width] with dense rows")
    M, K = t.shape
    return device, M, K, t.stride(0) if M > 1 else K


def mq_quantize8(x, codes_out=None, scales_out=None, stream=None):
    """(codes, scales): the rows of x [M, K] float16 in 8 bits. Enqueued on `stream` (no sync)."""
    device, M, K, xs = _half_matrix(x, "x")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_quantize8(x, codes_out, scales_out, stream)
    other = None if stream is None else _other(stream, x.device)
    codes_out, scales_out, cp, cs, sp, ss = _rows8_out(codes_out, scales_out, x, other, device)
    if M:
        code = lib.mq_quantize8(x.data_ptr(), M, K, xs, cp, cs, sp, ss, _stream(stream, device))
        if code:
            raise MQError(code, "mq_quantize8")
    return codes_out, scales_out


class Packed8:
    """A layer's weights in 8 bits (mq_w8 in include/mosaicq_head.h): the tensors of its codes and scales, uint8, in the
    order in which the matrix cores take them."""

    def __init__(self, codes, scales, N: int, K: int):
        self.N, self.K = int(N), int(K)
        nc, ns = _size(), _size()
        _check(lib.mq_pack8_bytes(self.N, self.K, ctypes.byref(nc), ctypes.byref(ns)), "mq_pack8_bytes")
        for t, name, n in ((codes, "codes", nc.value), (scales, "scales", ns.value)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.uint8 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous uint8 tensor on the GPU")
            if t.numel() != n:
                raise ValueError(f"{name} must hold {n} bytes")
        if scales.get_device() != codes.get_device():
            raise _apart("scales")
        self.codes, self.scales = codes, scales
        self.device = codes.get_device()
        self.device_bytes = nc.value + ns.value
        self._c = _W8(codes.data_ptr(), scales.data_ptr(), self.N, self.K)
        self._ref = ctypes.addressof(self._c)
        self._ws = {}      # tokens -> workspace bytes
        self._like = codes.new_empty(0, dtype=_F16)


def mq_pack8(W, stream=None) -> Packed8:
    """The weights W [N, K] float16 (rows may lie apart) in 8 bits. Enqueued on `stream` (no sync); a weight that is not
    finite makes its output feature NaN."""
    device, N, K, ws = _half_matrix(W, "W")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_pack8(W, stream)
    nc, ns = _size(), _size()
    _check(lib.mq_pack8_bytes(N, K, ctypes.byref(nc), ctypes.byref(ns)), "mq_pack8")
    other = None if stream is None else _other(stream, W.device)
    p = Packed8(*[_new(other, torch.empty, n.value, dtype=torch.uint8, device=W.device) for n in (nc, ns)], N, K)
    _check(lib.mq_pack8(W.data_ptr(), ws, p._ref, _stream(stream, device)), "mq_pack8")
    return p


def linear8_workspace(p: Packed8, tokens: int) -> int:
    """Bytes of workspace mq_linear8 needs for so many tokens."""
    n = p._ws.get(tokens)
    if n is None:
        out = _size()
        _check(lib.mq_linear8_workspace(tokens, p._ref, ctypes.byref(out)), "mq_linear8_workspace")
        n = p._ws[tokens] = out.value
    return n


def _workspace(workspace, need: int, device: int, other):
    """The tensor, address and bytes of a call's workspace: the given one, or one from the stream's pool."""
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != device or not workspace.is_contiguous():
            raise TypeError(f"workspace must be a contiguous uint8 tensor on GPU {device}")
        return workspace, workspace.data_ptr(), workspace.numel()
    if not need:
        return None, None, 0
    ws = _new(other, torch.empty, need, dtype=torch.uint8, device=torch.device("cuda", device))
    return ws, ws.data_ptr(), need


def mq_linear8(codes, scales, p: Packed8, out=None, workspace=None, stream=None):
    """Y [M, N] float16 of the 8-bit rows (codes, scales) [M, K] and the layer p. workspace: a uint8 GPU tensor of at
    least linear8_workspace bytes (None: taken from torch's allocator). Enqueued on `stream` (no sync)."""
    device = _device(codes, "codes", _E4M3)
    if p.device != device:
        raise _apart("p")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_linear8(codes, scales, p, out, workspace, stream)
    if codes.dim() != 2:
        raise ValueError("codes must be [tokens, 128 n]")
    M = codes.shape[0]
    cp, cs, sp, ss = _rows8(codes, scales, device, M, p.K)
    other = None if stream is None else _other(stream, codes.device)
    if out is None:
        out = _new(other, p._like.new_empty, (M, p.N))
        yp, ys = out.data_ptr(), p.N
    else:
        yp, ys = _matrix(out, "out", device, _F16, (M, p.N))
    if M == 0:
        return out
    ws, wp, nw = _workspace(workspace, linear8_workspace(p, M), device, other)
    code = lib.mq_linear8(cp, cs, sp, ss, M, p._ref, yp, ys, wp, nw, _stream(stream, device))
    if code:
        raise MQError(code, "mq_linear8")
    return out


_ws_sample = {}      # (rows, vocab, fp32) -> workspace bytes


def sample_workspace(rows: int, vocab: int, fp32: bool = False) -> int:
    """Bytes of workspace mq_sample needs for logits [rows, vocab]."""
    key = (rows, vocab, bool(fp32))
    n = _ws_sample.get(key)
    if n is None:
        out = _size()
        a = _SampleArgs(rows=rows, vocab=vocab, logits_fp32=int(fp32))
        _check(lib.mq_sample_workspace(ctypes.byref(a), ctypes.byref(out)), "mq_sample_workspace")
        n = _ws_sample[key] = out.value
    return n


def _setting(t, name: str, device: int, dt, rows: int) -> int:
    """Address of a row setting [rows], 0 where there is none."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not dt or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dt} tensor on GPU {device}")
    if t.dim() != 1 or t.shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}]")
    return t.data_ptr()


def mq_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, token_out=None, logprob_out=None,
              workspace=None, stream=None):
    """(token int32 [rows], logprob float32 [rows]): a token for each row of logits [rows, vocab] (float16 or float32)
    from uniform numbers u [rows] float32, under temperature, top_k (int32), top_p and min_p, each [rows] on the GPU or
    None (1, and no limit). logits may be one row that is expanded (many draws from it). See mq_sample in
    include/mosaicq_head.h. Enqueued on `stream` (no sync)."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype not in (_F16, torch.float32):
        raise TypeError("logits must be a float16 or float32 tensor on the GPU")
    device = logits.get_device()
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_sample(logits, u, temperature, top_k, top_p, min_p, token_out, logprob_out, workspace, stream)
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [rows, vocab] with dense rows")
    R, V = logits.shape
    f32 = torch.float32
    other = None if stream is None else _other(stream, logits.device)
    if u is None:
        raise TypeError("u must be a float32 tensor")
    up = _setting(u, "u", device, f32, R)
    settings = (_setting(temperature, "temperature", device, f32, R), _setting(top_k, "top_k", device, torch.int32, R),
                _setting(top_p, "top_p", device, f32, R), _setting(min_p, "min_p", device, f32, R))
    if token_out is None:
        token_out = _new(other, torch.empty_like, u, dtype=torch.int32)
    if logprob_out is None:
        logprob_out = _new(other, torch.empty_like, u)
    tp, lp = _setting(token_out, "token_out", device, torch.int32, R), _setting(logprob_out, "logprob_out", device, f32, R)
    if R == 0:
        return token_out, logprob_out
    fp32 = logits.dtype is f32
    ws, wp, nw = _workspace(workspace, sample_workspace(R, V, fp32), device, other)
    a = _sample_args(logits.data_ptr(), R, V, logits.stride(0) if R > 1 else V, *settings, up, tp, lp, fp32)
    code = lib.mq_sample(a, wp, nw, _stream(stream, device))
    if code:
        raise MQError(code, "mq_sample")
    return token_out, logprob_out
