"""The prompt operators on torch tensors: linear, gated_ffn, gated_ffn_backward, prompt_attention.

Thin wrappers of kd_linear, kd_gated_ffn, ... (include/kd.h): they check shapes, types and
devices, allocate the outputs (and the backward pass's workspace) with torch's allocator and
enqueue on the current stream of the tensors' device. Matrices may have any row stride that
is a multiple of 8 elements; their last dimension is contiguous. The functions record no
autograd graph: gated_ffn_backward returns the gradients.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import KdError, load_library as _lib

__all__ = ["linear", "gated_ffn", "gated_ffn_backward", "prompt_attention"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACT = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
# the C structs of kd.h, field by field
_LINEAR = struct.Struct("@4i3qPqPqPPqPq")
_GATED = struct.Struct("@2i3qPqPqPq")
_ATTENTION = struct.Struct("@4i2q" + "P2q" * 4 + "fPN")
_FEW_ROWS = 128 * 148  # query rows (tokens x heads) above which attention needs no workspace
_EINVAL = -1
# The current device and its current stream as plain numbers: the public calls build objects, which
# costs a call of a few microseconds a fifth of its time.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _refuse(text):
    raise KdError(_EINVAL, text)


def _check(rc):
    if rc:
        raise KdError(rc, (_lib().kd_op_error() or b"").decode())


def _act_id(act):
    try:
        return _ACT[act]
    except (KeyError, TypeError):
        _refuse("act must be one of none, relu, silu, gelu: got %r" % (act,))


def _wrong(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        _refuse("%s must be a tensor: got %s" % (name, type(t).__name__))
    _refuse("%s must be a %s tensor of shape %s on cuda:%d, the last dimension contiguous: got %s of shape %s, strides %s, on %s"
            % (name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), t.stride(), t.device))


def _matrix(name, t, shape, dtype, dev):
    """Checks a matrix of that shape and type on cuda:dev; returns its row stride."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            s0, s1 = t.stride()
            if s1 == 1 or shape[1] <= 1:
                return s0
    except (AttributeError, TypeError, ValueError):
        pass
    _wrong(name, t, shape, dtype, dev)


def _input(name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        _refuse("%s must be a 2-D CUDA tensor" % name)
    dtype = t.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        _refuse("%s must be bfloat16 or float16: got %s" % (name, dtype))
    return dtype, t.get_device()


def _columns(name, t, i):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse("%s must be a 2-D tensor" % name)
    return t.shape[i]


def _enqueue(dev, fn, *args):
    """Calls fn(*args, stream) with cuda:dev current; raises on an error code."""
    if dev == _device():
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    if rc:
        _check(rc)


def _empty(like, shape, dtype):
    """An output on like's device."""
    return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)


def linear(x, w, bias=None, act="none", residual=None, out=None, out_dtype=None, w_t=False):
    """residual + act(x @ w.T + bias) for x [m, k] and w [n, k] (w [k, n] with w_t).

    bias [n] has x's type; residual and out [m, n] have out_dtype: x's type (the default) or
    float32. act: none, relu, silu, gelu. residual may be out itself."""
    dtype, dev = _input("x", x)
    m, k = x.shape
    n = _columns("w", w, 1 if w_t else 0)
    ldx = _matrix("x", x, (m, k), dtype, dev)
    ldw = _matrix("w", w, (k, n) if w_t else (n, k), dtype, dev)
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        _refuse("out_dtype must be %s or torch.float32: got %s" % (dtype, out_dtype))
    if out is None:
        out, ldo = _empty(x, (m, n), out_dtype), n
    else:
        ldo = _matrix("out", out, (m, n), out_dtype, dev)
    pb = pr = ldr = 0
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.shape != (n,) or bias.dtype is not dtype or \
                bias.get_device() != dev or (n > 1 and bias.stride(0) != 1):
            _refuse("bias must be a contiguous (%d,) %s tensor on cuda:%d" % (n, dtype, dev))
        pb = bias.data_ptr()
    if residual is not None:
        ldr = _matrix("residual", residual, (m, n), out_dtype, dev)
        pr = residual.data_ptr()
    _enqueue(dev, _lib().kd_linear,
             _LINEAR.pack(_DTYPE[dtype], _DTYPE[out_dtype], _act_id(act), 1 if w_t else 0, m, n, k, x.data_ptr(), ldx,
                          w.data_ptr(), ldw, pb, pr, ldr, out.data_ptr(), ldo))
    return out


def _gated(x, wg, wu, act):
    dtype, dev = _input("x", x)
    m, d = x.shape
    f = _columns("wg", wg, 0)
    args = _GATED.pack(_DTYPE[dtype], _act_id(act), m, d, f, x.data_ptr(), _matrix("x", x, (m, d), dtype, dev),
                       wg.data_ptr(), _matrix("wg", wg, (f, d), dtype, dev), wu.data_ptr(),
                       _matrix("wu", wu, (f, d), dtype, dev))
    return args, dtype, dev, m, d, f


def gated_ffn(x, wg, wu, act="silu", out=None):
    """act(x @ wg.T) * (x @ wu.T) for x [m, d], wg and wu [f, d] (rows may be interleaved)."""
    args, dtype, dev, m, d, f = _gated(x, wg, wu, act)
    if out is None:
        out, ldo = _empty(x, (m, f), dtype), f
    else:
        ldo = _matrix("out", out, (m, f), dtype, dev)
    _enqueue(dev, _lib().kd_gated_ffn, args, out.data_ptr(), ldo)
    return out


def gated_ffn_backward(x, wg, wu, dh, act="silu"):
    """(dx, dwg, dwu) of gated_ffn for the gradient dh [m, f] of its result."""
    args, dtype, dev, m, d, f = _gated(x, wg, wu, act)
    ldh = _matrix("dh", dh, (m, f), dtype, dev)
    dx, dwg, dwu = _empty(x, (m, d), dtype), _empty(x, (f, d), dtype), _empty(x, (f, d), dtype)
    if m == 0 or f == 0:  # sums over nothing
        return dx.zero_(), dwg.zero_(), dwu.zero_()
    lib = _lib()
    n = lib.kd_gated_ffn_backward_workspace(m, f)
    ws = _empty(x, (n,), torch.uint8)
    _enqueue(dev, lib.kd_gated_ffn_backward, args, dh.data_ptr(), ldh, dx.data_ptr(), d, dwg.data_ptr(), d,
             dwu.data_ptr(), d, ws.data_ptr(), n)
    return dx, dwg, dwu


def prompt_attention(q, k, v, kv_len, scale=None, out=None):
    """Causal attention of the n new tokens q [n, heads, hd] over a cache k, v [kv_heads, S, hd].

    The cache holds kv_len earlier positions and the n new ones (S >= kv_len + n); token i sees
    the positions up to kv_len + i. scale: 1 / sqrt(hd) unless given. v has to be finite at
    all kv_len + n positions; what lies behind them is not read."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not q.is_cuda:
        _refuse("q must be a 3-D CUDA tensor [n, heads, head_dim]")
    dtype, dev = q.dtype, q.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        _refuse("q must be bfloat16 or float16: got %s" % (dtype,))
    n, hq, hd = q.shape
    kv_len = int(kv_len)
    if kv_len < 0:
        _refuse("kv_len must not be negative")
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype is not dtype or t.get_device() != dev:
            _refuse("%s must be a 3-D %s tensor on cuda:%d" % (name, dtype, dev))
        shape = t.shape
        if shape[2] != hd or shape[0] != k.shape[0] or shape[1] < kv_len + n:
            _refuse("%s has shape %s: need [%d, >= %d, %d]" % (name, tuple(shape), k.shape[0], kv_len + n, hd))
    if out is None:
        out = _empty(q, (n, hq, hd), dtype)
    elif not isinstance(out, torch.Tensor) or out.shape != q.shape or out.dtype is not dtype or out.get_device() != dev:
        _refuse("out must be a %s tensor of q's shape on cuda:%d" % (dtype, dev))
    if scale is None:
        scale = hd ** -0.5
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    if qs[2] != 1 or ks[2] != 1 or vs[2] != 1 or os[2] != 1:
        _refuse("the last dimension must be contiguous")
    lib = _lib()
    args = (_DTYPE[dtype], hq, k.shape[0], hd, n, kv_len, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[1], ks[0],
            v.data_ptr(), vs[1], vs[0], out.data_ptr(), os[0], os[1], scale)
    size, ws = 0, 0
    if n * hq <= _FEW_ROWS:  # only few tiles are split
        size = lib.kd_prompt_attention_workspace(_ATTENTION.pack(*args, 0, 0))
        if size:
            buf = _empty(q, (size,), torch.uint8)  # returned to the allocator in stream order
            ws = buf.data_ptr()
    _enqueue(dev, lib.kd_prompt_attention, _ATTENTION.pack(*args, ws, size))
    return out
