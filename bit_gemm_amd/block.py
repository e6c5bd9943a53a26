"""Python binding of include/mosaicq_block.h (ctypes): the operators between a
decoder block's 4-bit linears.

    rope = Rope(128, positions=32768)                       # cos/sin table
    cache = KVCache.empty(blocks, slots, kv_heads, 128)     # 8-bit blocks and fp16 tails
    batch = KVBatch(cu_q, kv_len, block_table, max_new, max_len, slots=slots)
    q = mq_kv_append(q, k, v, cache, batch, rope=rope)      # rotates q and k, writes k and v
    o = mq_kv_attention(q, cache, batch)
    r, h = mq_norm_residual(y, r, w_pre)                    # r' = r + y, h = norm(r') w_pre
    r, codes, scales = mq_norm_residual_q8(y, r, w_pre)     # h as 8-bit rows, for head.mq_linear8

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

from .mosaicq import MQError, STATUS, _check, _new, _other  # noqa: F401  (the errors of both libraries are the same)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmosaicq_block.so")

BLOCK = 64                                      # tokens of a cache block
FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class _RopeSpec(ctypes.Structure):
    _fields_ = [("rot_dim", _i32), ("scaling", _i32)] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "original", "turns_fast", "turns_slow")]


class _RopePlan(ctypes.Structure):
    _fields_ = [("table", _vp), ("positions", _i64), ("rot_dim", _i32), ("layout", _i32)]


class _Cache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")] + [
        ("num_blocks", _i64), ("num_slots", _i64), ("kv_heads", _i32), ("head_dim", _i32), ("format", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("cu_q", "kv_len", "block_table", "slots")] + [
        (n, _i64) for n in ("seqs", "tokens", "table_width", "max_new", "max_len")]


class _NormArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("y", "r", "gate", "w_post", "w_pre", "r_out", "h_out")] + [
        (n, _i64) for n in ("tokens", "width", "y_stride", "r_stride", "gate_stride", "r_out_stride", "h_stride")] + [
        (n, _f32) for n in ("alpha", "beta", "eps", "weight_offset")] + [("residual_fp32", _i32)]


# the same fields in their order, packed in a fifth of the time that the structure takes
_norm_args = struct.Struct("@7P7q4fi4x").pack
_batch_args = struct.Struct("@4P5q").pack

EXPORTED = ("mq_rope_table", "mq_rope", "mq_kv_append", "mq_kv_attention", "mq_kv_attention_workspace",
            "mq_norm_residual", "mq_norm_residual_q8")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built (run `python -m bit_gemm_amd.build`)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.mq_rope_table.argtypes = [_vp, _i64, _vp, _vp]
    lib.mq_rope.argtypes = [_vp, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _i64, _vp]
    lib.mq_kv_append.argtypes = [_vp, _vp, _vp, _i32, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp]
    lib.mq_kv_attention_workspace.argtypes = [_vp, _vp, _i32, _vp]
    lib.mq_kv_attention.argtypes = [_vp, _vp, _vp, _i32, _i64, _i32, _f32, _vp, _i64, _vp, ctypes.c_size_t, _vp]
    lib.mq_norm_residual.argtypes = [_vp, _vp]
    lib.mq_norm_residual_q8.argtypes = [_vp, _vp, _i64, _vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()
_F16 = torch.float16


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without the Python object around it, where torch has that (3 us less a call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, device: int) -> int:
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _like(t):
    """A dense tensor of t's shape and type (0.6 us faster than by shape, where t is dense)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _device(t, name: str, dt) -> int:
    """The device of a call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dt:
        raise TypeError(f"{name} must be a {dt} tensor on the GPU")
    return t.get_device()


def _apart(name: str):
    return ValueError(f"{name} is on another device than the call's tensors")


def _rows(t, name: str, device: int, heads=None, dim=None):
    """Checks an fp16 [tokens, heads, dim] tensor on the device whose heads lie
    dense in a row; gives its tokens, heads and the elements between rows (of at
    most one row: its own width, whatever its stride says)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not _F16:
        raise TypeError(f"{name} must be a float16 tensor on GPU {device}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim or 'head dim'}]")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (H > 1 and sh != D):
        raise ValueError(f"the heads of a row of {name} must be dense")
    return T, H, st if T > 1 else H * D


def _ints(t, name: str, device: int, shape):
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor on GPU {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")
    return t


class Rope:
    """Cosines and sines of positions 0 .. positions - 1 for `rot_dim` rotated
    elements (see mq_rope_table in include/mosaicq_block.h); scaling "none",
    "linear", "base" or "parts"."""

    def __init__(self, rot_dim: int, positions: int, layout: str = "half", theta: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original: float = 8192.0, turns_fast: float = 32.0,
                 turns_slow: float = 1.0, stream=None):
        if layout not in LAYOUTS or scaling not in SCALINGS:
            raise ValueError(f"layout is one of {list(LAYOUTS)}, scaling one of {list(SCALINGS)}")
        self.rot_dim, self.positions, self.layout = int(rot_dim), int(positions), layout
        spec = _RopeSpec(self.rot_dim, SCALINGS[scaling], theta, factor, original, turns_fast, turns_slow)
        shape = (max(self.positions, 1), max(self.rot_dim // 2, 1), 2)
        other = None if stream is None else _other(stream)
        self.table = _new(other, torch.empty, shape, dtype=torch.float32, device="cuda")
        self.device = self.table.get_device()
        _check(lib.mq_rope_table(ctypes.byref(spec), self.positions, self.table.data_ptr(),
                                 _stream(stream, self.device)), "mq_rope_table")
        self._plan = _RopePlan(self.table.data_ptr(), self.positions, self.rot_dim, LAYOUTS[layout])
        self._ref = ctypes.addressof(self._plan)


def mq_rope(x, rope: Rope, pos, inverse: bool = False, out=None, stream=None):
    """x [tokens, heads, head_dim] with its heads turned to positions pos
    [tokens] int32 (turned back with inverse); out may be x. Enqueued on
    `stream` (no sync)."""
    device = _device(x, "x", _F16)
    if rope.device != device:
        raise _apart("rope")
    if x.dim() != 3 or x.stride(2) != 1:
        raise ValueError("x must be [tokens, heads, head_dim] with dense heads")
    T, H, D = x.shape
    _ints(pos, "pos", device, (T,))
    if out is not None and (out.dtype is not _F16 or out.get_device() != device or out.shape != x.shape or
                            out.stride(2) != 1):
        raise ValueError("out must be a float16 tensor of x's shape with dense heads, on x's device")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_rope(x, rope, pos, inverse, out, stream)
    if out is None:
        out = _like(x) if stream is None else _new(_other(stream, x.device), _like, x)
    if T == 0:
        return out
    xt, xh, _ = x.stride()
    yt, yh, _ = out.stride()
    code = lib.mq_rope(x.data_ptr(), T, H, D, xt, xh, pos.data_ptr(), rope._ref, int(inverse), out.data_ptr(), yt, yh,
                       _stream(stream, device))
    if code:
        raise MQError(code, "mq_rope")
    return out


class KVCache:
    """A key/value cache in 8 bits: the tensors of mq_kv_cache (see
    include/mosaicq_block.h). Codes are int8 or float8_e4m3fn."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, k_tail, v_tail):
        if k_codes.dtype not in FORMATS or v_codes.dtype is not k_codes.dtype:
            raise TypeError("codes must be int8 or float8_e4m3fn tensors")
        if k_codes.dim() != 4 or k_codes.shape[2] != BLOCK:
            raise ValueError(f"k_codes must be [blocks, kv_heads, {BLOCK}, head_dim]")
        nb, hk, _, D = k_codes.shape
        if k_tail.dim() != 4:
            raise ValueError(f"k_tail must be [slots, kv_heads, {BLOCK}, head_dim]")
        ns = k_tail.shape[0]
        want = {"k_codes": (k_codes, k_codes.dtype, (nb, hk, BLOCK, D)), "v_codes": (v_codes, k_codes.dtype, (nb, hk, D, BLOCK)),
                "k_scale": (k_scale, torch.float32, (nb, hk)), "v_scale": (v_scale, torch.float32, (nb, hk)),
                "k_tail": (k_tail, _F16, (ns, hk, BLOCK, D)), "v_tail": (v_tail, _F16, (ns, hk, D, BLOCK))}
        for name, (t, dt, shape) in want.items():
            if not t.is_cuda or t.dtype is not dt or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous {dt} tensor on the GPU")
            if t.get_device() != k_codes.get_device():
                raise ValueError(f"{name} must be on the device of k_codes")
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.k_tail, self.v_tail = k_tail, v_tail
        self.num_blocks, self.num_slots, self.kv_heads, self.head_dim = nb, ns, hk, D
        self.device = k_codes.get_device()
        self._c = _Cache(*[t.data_ptr() for t in (k_codes, v_codes, k_scale, v_scale, k_tail, v_tail)], nb, ns, hk, D,
                         FORMATS[k_codes.dtype])
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, blocks: int, slots: int, kv_heads: int, head_dim: int, fmt: str = "int8", device="cuda"):
        """A cache of `blocks` blocks and `slots` tails, zeroed."""
        dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
        def z(shape, t):
            return torch.zeros(shape, dtype=t, device=device)
        return cls(z((blocks, kv_heads, BLOCK, head_dim), torch.int8).view(dt),
                   z((blocks, kv_heads, head_dim, BLOCK), torch.int8).view(dt),
                   z((blocks, kv_heads), torch.float32), z((blocks, kv_heads), torch.float32),
                   z((slots, kv_heads, BLOCK, head_dim), _F16), z((slots, kv_heads, head_dim, BLOCK), _F16))


class KVBatch:
    """The sequences of one step (mq_kv_batch): cu_q [seqs + 1] where each
    sequence's new tokens start, kv_len [seqs] its tokens with the new ones,
    block_table [seqs, width] its cache blocks, slots [seqs] its tail slot
    (None: the sequence's own number), all int32 on the GPU and read when the
    kernels run. max_new and max_len bound what they hold."""

    def __init__(self, cu_q, kv_len, block_table, max_new: int, max_len: int, slots=None):
        S = kv_len.shape[0]
        self.device = _device(cu_q, "cu_q", torch.int32)
        self.cu_q, self.kv_len = _ints(cu_q, "cu_q", self.device, (S + 1,)), _ints(kv_len, "kv_len", self.device, (S,))
        if block_table.dim() != 2:
            raise ValueError("block_table must be [seqs, width]")
        self.block_table = _ints(block_table, "block_table", self.device, (S, block_table.shape[1]))
        self.slots = None if slots is None else _ints(slots, "slots", self.device, (S,))
        self.seqs, self.max_new, self.max_len = S, int(max_new), int(max_len)
        self._head = (cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                      0 if slots is None else slots.data_ptr(), S)
        self._rest = (block_table.shape[1], self.max_new, self.max_len)
        self._ws = {}      # (tokens, q heads, kv heads, head dim) -> workspace bytes

    def _with(self, tokens: int) -> bytes:
        """The mq_kv_batch of a call of so many tokens: each call's own, since calls may run in several threads."""
        return _batch_args(*self._head, tokens, *self._rest)


def mq_kv_append(q, k, v, cache: KVCache, batch: KVBatch, rope: Rope | None = None, q_out=None, stream=None):
    """Writes the new tokens' k and v [tokens, kv_heads, head_dim] into the
    cache. With a rope plan keys are turned to their positions first, and so
    are the queries q [tokens, q_heads, head_dim] (None: no queries), which
    are returned (in q_out where given; it may be q). Without one q is returned
    as it is, and there is no q_out. Rows may lie apart (slices of a joined
    projection). Enqueued on `stream` (no sync)."""
    D, hk, device = cache.head_dim, cache.kv_heads, cache.device
    T, _, ks = _rows(k, "k", device, hk, D)
    Tv, _, vs = _rows(v, "v", device, hk, D)
    if batch.device != device:
        raise _apart("batch")
    if Tv != T:
        raise ValueError("k and v must have the same tokens")
    if q_out is not None and q_out is not q and (q is None or rope is None):
        raise ValueError("q_out is written with queries and a rope plan only")
    qp = qo = rp = None
    heads = qs = qos = 0
    if rope is not None:
        if rope.device != device:
            raise _apart("rope")
        rp = rope._ref
        if q is not None:
            Tq, heads, qs = _rows(q, "q", device, None, D)
            To, _, qos = _rows(q_out, "q_out", device, heads, D) if q_out is not None else (Tq, heads, heads * D)
            if Tq != T or To != T:
                raise ValueError("q, q_out, k and v must have the same tokens")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_kv_append(q, k, v, cache, batch, rope, q_out, stream)
    if heads:
        if q_out is None:
            q_out = _like(q) if stream is None else _new(_other(stream, q.device), _like, q)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    if T:
        code = lib.mq_kv_append(cache._ref, batch._with(T), qp, heads, qs, k.data_ptr(), ks, v.data_ptr(), vs, rp, qo,
                                qos, _stream(stream, device))
        if code:
            raise MQError(code, "mq_kv_append")
    return q if qo is None else q_out


def kv_attention_workspace(cache: KVCache, batch: KVBatch, tokens: int, q_heads: int) -> int:
    """Bytes of workspace mq_kv_attention needs for these sizes."""
    key = (tokens, q_heads, cache.kv_heads, cache.head_dim)
    n = batch._ws.get(key)
    if n is None:
        out = ctypes.c_size_t()
        _check(lib.mq_kv_attention_workspace(cache._ref, batch._with(tokens), q_heads, ctypes.byref(out)),
               "mq_kv_attention_workspace")
        n = batch._ws[key] = out.value
    return n


def mq_kv_attention(q, cache: KVCache, batch: KVBatch, causal: bool = True, scale: float | None = None, out=None,
                    workspace=None, stream=None):
    """softmax(scale q k^T) v of q [tokens, q_heads, head_dim] over the cache
    (scale: head_dim^-1/2 by default), causal with the last new token at the
    sequence's end, or over all cached tokens. workspace: a uint8 GPU tensor of
    at least kv_attention_workspace bytes (None: taken from torch's allocator).
    Enqueued on `stream` (no sync)."""
    D, device = cache.head_dim, cache.device
    T, H, qs = _rows(q, "q", device, None, D)
    if batch.device != device:
        raise _apart("batch")
    os_ = H * D
    if out is not None:
        To, _, os_ = _rows(out, "out", device, H, D)
        if To != T:
            raise ValueError("out must have q's tokens")
    if workspace is not None and (workspace.dtype is not torch.uint8 or workspace.get_device() != device or
                                  not workspace.is_contiguous()):
        raise TypeError(f"workspace must be a contiguous uint8 tensor on GPU {device}")
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_kv_attention(q, cache, batch, causal, scale, out, workspace, stream)
    other = None if stream is None else _other(stream, q.device)
    if out is None:
        out = _new(other, _like, q)
    if T == 0:
        return out
    need = kv_attention_workspace(cache, batch, T, H)
    wp, nw = None, 0
    if workspace is not None:
        wp, nw = workspace.data_ptr(), workspace.numel()
    elif need:
        ws = _new(other, torch.empty, need, dtype=torch.uint8, device=q.device)
        wp, nw = ws.data_ptr(), need
    code = lib.mq_kv_attention(cache._ref, batch._with(T), q.data_ptr(), H, qs, int(causal),
                               D ** -0.5 if scale is None else scale, out.data_ptr(), os_, wp, nw,
                               _stream(stream, device))
    if code:
        raise MQError(code, "mq_kv_attention")
    return out


def _matrix(t, name: str, device: int, dt, shape):
    """Address and row stride of a [tokens, width] tensor on the device with dense rows."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not dt:
        raise TypeError(f"{name} must be a {dt} tensor on GPU {device}")
    st = t.stride()
    if t.shape != shape or st[1] != 1:
        raise ValueError(f"{name} must be {list(shape)} with dense rows")
    return t.data_ptr(), st[0] if shape[0] > 1 else shape[1]


def _vector(t, name: str, device: int, width: int):
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not _F16 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float16 tensor on GPU {device}")
    if t.dim() != 1 or t.shape[0] != width:
        raise ValueError(f"{name} must be [{width}]")
    return t.data_ptr()


def _branch(y, r, w_post, gate, r_out, other, device: int, shape, dt):
    """Addresses and strides of a norm's branch: y, w_post, gate and r_out, which is made where it is not given."""
    M, W = shape
    yp, ys = _matrix(y, "y", device, _F16, shape)
    wpost = gp = gs = 0
    if r_out is None:
        r_out = _new(other, _like, r)
        rp, rs = r_out.data_ptr(), W
    else:
        rp, rs = _matrix(r_out, "r_out", device, dt, shape)
    if w_post is not None:
        wpost = _vector(w_post, "w_post", device, W)
    if gate is not None:
        if gate.dim() == 1:
            gp = _vector(gate, "gate", device, W)
        else:
            gp, gs = _matrix(gate, "gate", device, _F16, shape)
    return yp, ys, wpost, gp, gs, r_out, rp, rs


def mq_norm_residual(y, r, w_pre, w_post=None, gate=None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                     weight_offset: float = 0.0, r_out=None, h_out=None, stream=None):
    """(r', h): r' = alpha r + beta gate N(y) and h = norm(r') (w_pre + offset),
    N the norm with w_post (None: the branch as it is). y None: r' is r and
    only h is made; w_pre None: only r' is made (h is None). y [tokens, width]
    float16, r float16 or float32, gate [tokens, width] (expanded over tokens
    where all share it) or [width]; r_out may be r. Enqueued on `stream` (no
    sync)."""
    if not isinstance(r, torch.Tensor) or not r.is_cuda or r.dtype not in (_F16, torch.float32):
        raise TypeError("r must be a float16 or float32 tensor on the GPU")
    device = r.get_device()
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_norm_residual(y, r, w_pre, w_post, gate, alpha, beta, eps, weight_offset, r_out, h_out, stream)
    if r.dim() != 2 or r.stride(1) != 1:
        raise ValueError("r must be [tokens, width] with dense rows")
    shape, dt = r.shape, r.dtype
    M, W = shape
    other = None if stream is None else _other(stream, r.device)
    yp = gp = rp = hp = wpost = wpre = ys = gs = rs = hs = 0
    if y is not None:
        yp, ys, wpost, gp, gs, r_out, rp, rs = _branch(y, r, w_post, gate, r_out, other, device, shape, dt)
    else:
        r_out = r
    if w_pre is not None:
        wpre = _vector(w_pre, "w_pre", device, W)
        if h_out is None:
            h_out = _new(other, w_pre.new_empty, shape) if y is None else _new(other, _like, y)
            hp, hs = h_out.data_ptr(), W
        else:
            hp, hs = _matrix(h_out, "h_out", device, _F16, shape)
    else:
        h_out = None
    if M == 0:
        return r_out, h_out
    a = _norm_args(yp, r.data_ptr(), gp, wpost, wpre, rp, hp, M, W, ys, r.stride(0) if M > 1 else W, gs, rs, hs, alpha,
                   beta, eps, weight_offset, dt is not _F16)
    code = lib.mq_norm_residual(a, _stream(stream, device))
    if code:
        raise MQError(code, "mq_norm_residual")
    return r_out, h_out


_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _rows8(codes, scales, device: int, tokens: int, width: int):
    """Checks the 8-bit rows of [tokens, width]: codes float8_e4m3fn [tokens, 128 n], scales float8_e8m0fnu [tokens, n],
    n = ceil(width / 128), rows dense. Addresses and strides."""
    n = (width + 127) // 128
    cp, cs = _matrix(codes, "codes", device, _E4M3, (tokens, 128 * n))
    sp, ss = _matrix(scales, "scales", device, _E8M0, (tokens, n))
    return cp, cs, sp, ss


def _rows8_out(codes, scales, x, other, device: int):
    """The 8-bit rows that a call writes for x [tokens, width], made where they are not given; addresses and strides."""
    M, W = x.shape
    n = (W + 127) // 128
    if codes is None:        # by empty_like where it is x's shape (0.5 us faster)
        codes = (_new(other, torch.empty_like, x, dtype=_E4M3) if W == 128 * n and x.is_contiguous() else
                 _new(other, x.new_empty, (M, 128 * n), dtype=_E4M3))
        cp, cs = codes.data_ptr(), 128 * n
    else:
        cp, cs = _matrix(codes, "codes", device, _E4M3, (M, 128 * n))
    if scales is None:
        scales = _new(other, x.new_empty, (M, n), dtype=_E8M0)
        sp, ss = scales.data_ptr(), n
    else:
        sp, ss = _matrix(scales, "scales", device, _E8M0, (M, n))
    return codes, scales, cp, cs, sp, ss


def mq_norm_residual_q8(y, r, w_pre, w_post=None, gate=None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                        weight_offset: float = 0.0, r_out=None, codes_out=None, scales_out=None, stream=None):
    """(r', codes, scales): mq_norm_residual with h = norm(r') (w_pre + offset) as 8-bit rows, for head.mq_linear8.
    codes float8_e4m3fn [tokens, 128 n] and scales float8_e8m0fnu [tokens, n], n = ceil(width / 128): a power of two
    for each block of 128 elements, zeros past width (all codes of a block with an Inf or NaN are NaN, its scale too).
    Enqueued on `stream` (no sync)."""
    if not isinstance(r, torch.Tensor) or not r.is_cuda or r.dtype not in (_F16, torch.float32):
        raise TypeError("r must be a float16 or float32 tensor on the GPU")
    device = r.get_device()
    if device != _current_device():
        with torch.cuda.device(device):
            return mq_norm_residual_q8(y, r, w_pre, w_post, gate, alpha, beta, eps, weight_offset, r_out, codes_out,
                                       scales_out, stream)
    if r.dim() != 2 or r.stride(1) != 1:
        raise ValueError("r must be [tokens, width] with dense rows")
    shape, dt = r.shape, r.dtype
    M, W = shape
    other = None if stream is None else _other(stream, r.device)
    yp = gp = rp = wpost = ys = gs = rs = 0
    if y is not None:
        yp, ys, wpost, gp, gs, r_out, rp, rs = _branch(y, r, w_post, gate, r_out, other, device, shape, dt)
    else:
        r_out = r
    wpre = _vector(w_pre, "w_pre", device, W)
    codes_out, scales_out, cp, cs, sp, ss = _rows8_out(codes_out, scales_out, r, other, device)
    if M == 0:
        return r_out, codes_out, scales_out
    a = _norm_args(yp, r.data_ptr(), gp, wpost, wpre, rp, cp, M, W, ys, r.stride(0) if M > 1 else W, gs, rs, cs, alpha,
                   beta, eps, weight_offset, dt is not _F16)
    code = lib.mq_norm_residual_q8(a, sp, ss, _stream(stream, device))
    if code:
        raise MQError(code, "mq_norm_residual_q8")
    return r_out, codes_out, scales_out
