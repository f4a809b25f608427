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

from . import KdError, load_library

__all__ = ["linear", "gated_ffn", "gated_ffn_backward", "prompt_attention"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACT = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
# the C structs of kd.h, field by field
_LINEAR = struct.Struct("@4i3qPqPqPPqPq")
_GATED = struct.Struct("@2i3qPqPqPq")
_ATTENTION = struct.Struct("@4i2q" + "P2q" * 4 + "fi")
_EINVAL = -1


def _refuse(text):
    raise KdError(_EINVAL, text)


def _check(rc):
    if rc:
        raise KdError(rc, (load_library().kd_op_error() or b"").decode())


def _act_id(act):
    try:
        return _ACT[act]
    except (KeyError, TypeError):
        _refuse("act must be one of none, relu, silu, gelu: got %r" % (act,))


def _matrix(name, t, rows, cols, dtype, device):
    """Checks a [rows][cols] tensor of that type and device; returns its row stride."""
    if t.dim() != 2 or t.dtype is not dtype or t.device != device:
        _refuse("%s must be a 2-D %s tensor on %s: got %s %s on %s" % (name, dtype, device, tuple(t.shape), t.dtype, t.device))
    r, c = t.shape
    if r != rows or c != cols:
        _refuse("%s has shape (%d, %d), expected (%d, %d)" % (name, r, c, rows, cols))
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        _refuse("%s: the last dimension must be contiguous" % name)
    return s0


def _input(name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.device.type != "cuda":
        _refuse("%s must be a 2-D CUDA tensor" % name)
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
        _refuse("%s must be bfloat16 or float16: got %s" % (name, t.dtype))
    return t.dtype, t.device


def _enqueue(device, fn, *args):
    """Calls fn(*args, stream) with `device` current; raises on an error code."""
    i = device.index
    if i == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream(i).cuda_stream)
    else:
        with torch.cuda.device(i):
            rc = fn(*args, torch.cuda.current_stream(i).cuda_stream)
    if rc:
        _check(rc)


def linear(x, w, bias=None, act="none", residual=None, out=None, out_dtype=None, w_t=False):
    """residual + act(x @ w.T + bias) for x [m, k] and w [n, k] (w [k, n] with w_t).

    bias [n] has x's type; residual and out [m, n] have out_dtype: x's type (the default) or
    float32. act: none, relu, silu, gelu. residual may be out itself."""
    dtype, device = _input("x", x)
    m, k = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        _refuse("w must be a 2-D tensor")
    n = w.shape[1 if w_t else 0]
    ldx = _matrix("x", x, m, k, dtype, device)
    ldw = _matrix("w", w, k, n, dtype, device) if w_t else _matrix("w", w, n, k, dtype, device)
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        _refuse("out_dtype must be %s or torch.float32: got %s" % (dtype, out_dtype))
    if out is None:
        out, ldo = torch.empty((m, n), dtype=out_dtype, device=device), n
    else:
        ldo = _matrix("out", out, m, n, out_dtype, device)
    pb = 0
    if bias is not None:
        if bias.shape != (n,) or bias.dtype is not dtype or bias.device != device or (bias.stride(0) != 1 and n > 1):
            _refuse("bias must be a contiguous (%d,) %s tensor on %s" % (n, dtype, device))
        pb = bias.data_ptr()
    pr = ldr = 0
    if residual is not None:
        ldr = _matrix("residual", residual, m, n, out_dtype, device)
        pr = residual.data_ptr()
    _enqueue(device, load_library().kd_linear,
             _LINEAR.pack(_DTYPE[dtype], _DTYPE[out_dtype], _act_id(act), 1 if w_t else 0, m, n, k, x.data_ptr(), ldx,
                          w.data_ptr(), ldw, pb, pr, ldr, out.data_ptr(), ldo))
    return out


def _gated(x, wg, wu, act):
    dtype, device = _input("x", x)
    m, d = x.shape
    if not isinstance(wg, torch.Tensor) or wg.dim() != 2 or not isinstance(wu, torch.Tensor):
        _refuse("wg and wu must be 2-D tensors")
    f = wg.shape[0]
    args = _GATED.pack(_DTYPE[dtype], _act_id(act), m, d, f, x.data_ptr(), _matrix("x", x, m, d, dtype, device),
                       wg.data_ptr(), _matrix("wg", wg, f, d, dtype, device),
                       wu.data_ptr(), _matrix("wu", wu, f, d, dtype, device))
    return args, dtype, device, m, d, f


def gated_ffn(x, wg, wu, act="silu", out=None):
    """act(x @ wg.T) * (x @ wu.T) for x [m, d], wg and wu [f, d] (rows may be interleaved)."""
    args, dtype, device, m, d, f = _gated(x, wg, wu, act)
    if out is None:
        out, ldo = torch.empty((m, f), dtype=dtype, device=device), f
    else:
        ldo = _matrix("out", out, m, f, dtype, device)
    _enqueue(device, load_library().kd_gated_ffn, args, out.data_ptr(), ldo)
    return out


def gated_ffn_backward(x, wg, wu, dh, act="silu"):
    """(dx, dwg, dwu) of gated_ffn for the gradient dh [m, f] of its result."""
    args, dtype, device, m, d, f = _gated(x, wg, wu, act)
    ldh = _matrix("dh", dh, m, f, dtype, device)
    dx, dwg, dwu = (torch.empty(s, dtype=dtype, device=device) for s in ((m, d), (f, d), (f, d)))
    if m == 0 or f == 0:  # sums over nothing
        return dx.zero_(), dwg.zero_(), dwu.zero_()
    lib = load_library()
    n = lib.kd_gated_ffn_backward_workspace(m, f)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _enqueue(device, lib.kd_gated_ffn_backward, args, dh.data_ptr(), ldh, dx.data_ptr(), d, dwg.data_ptr(), d,
             dwu.data_ptr(), d, ws.data_ptr(), n)
    return dx, dwg, dwu


def prompt_attention(q, k, v, kv_len, scale=None, out=None):
    """Causal attention of the n new tokens q [n, heads, hd] over a cache k, v [kv_heads, S, hd].

    The cache holds kv_len earlier positions and the n new ones (S >= kv_len + n); token i sees
    the positions up to kv_len + i. scale: 1 / sqrt(hd) unless given. v has to be finite at
    all kv_len + n positions; what lies behind them is not read."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.device.type != "cuda":
        _refuse("q must be a 3-D CUDA tensor [n, heads, head_dim]")
    dtype, device = q.dtype, q.device
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        _refuse("q must be bfloat16 or float16: got %s" % (dtype,))
    n, hq, hd = q.shape
    kv_len = int(kv_len)
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype is not dtype or t.device != device:
            _refuse("%s must be a 3-D %s tensor on %s" % (name, dtype, device))
        if t.shape[2] != hd or t.shape[0] != k.shape[0] or t.shape[1] < kv_len + n:
            _refuse("%s has shape %s: need [%d, >= %d, %d]" % (name, tuple(t.shape), k.shape[0], kv_len + n, hd))
    if out is None:
        out = torch.empty((n, hq, hd), dtype=dtype, device=device)
    elif out.shape != q.shape or out.dtype is not dtype or out.device != device:
        _refuse("out must be a %s tensor of q's shape on %s" % (dtype, device))
    if kv_len < 0:
        _refuse("kv_len must not be negative")
    if scale is None:
        scale = hd ** -0.5
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    if qs[2] != 1 or ks[2] != 1 or vs[2] != 1 or os[2] != 1:
        _refuse("the last dimension must be contiguous")
    _enqueue(device, load_library().kd_prompt_attention,
             _ATTENTION.pack(_DTYPE[dtype], hq, k.shape[0], hd, n, kv_len, q.data_ptr(), qs[0], qs[1], k.data_ptr(),
                             ks[1], ks[0], v.data_ptr(), vs[1], vs[0], out.data_ptr(), os[0], os[1], scale, 0))
    return out
