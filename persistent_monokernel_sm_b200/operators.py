"""The prompt operators on torch tensors: linear, gated_ffn, gated_ffn_backward, prompt_attention.

They check shapes, types and devices, allocate outputs and workspaces with torch's allocator and
enqueue kd_linear, kd_gated_ffn, ... (include/kd.h) on the current stream of the tensors' device;
all of that is in csrc/kd_torch.cpp. Tensors are bfloat16 or float16 and their last dimension is
contiguous; rows of a product's inputs start on 16 bytes (a row stride that is a multiple of 8
elements). The functions record no autograd graph (gated_ffn_backward returns the gradients): where
gradients are enabled, tensors that require them are refused; torch.no_grad() or a
torch.autograd.Function around the calls is the way. An `out` counts as changed in place.

What they refuse raises KdError. A device-side wait that exceeds its limit (kd_op_set_timeout; none
comes near the default of 2 s) ends its kernel early with outputs that are not valid: kd_op_sync
waits for a stream and raises KdError (KD_ETIMEOUT) then.
"""

from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch  # noqa: F401  (its libraries have to be loaded first)

from . import LIB_PATH, KdError, load_library

__all__ = ["linear", "gated_ffn", "gated_ffn_backward", "prompt_attention"]


def _load():
    load_library()
    path = os.path.join(os.path.dirname(LIB_PATH), "_kd_torch.so")
    if not os.path.exists(path):
        raise ImportError("_kd_torch.so not found at %s; build it with persistent_monokernel_sm_b200/build.py" % path)
    spec = importlib.util.spec_from_loader("_kd_torch", importlib.machinery.ExtensionFileLoader("_kd_torch", path))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_error(KdError)
    return module


_t = _load()


def linear(x, w, bias=None, act="none", residual=None, out=None, out_dtype=None, w_t=False):
    """residual + act(x @ w.T + bias) for x [m, k] and w [n, k] (w [k, n] with w_t).

    bias [n] has x's type; residual and out [m, n] have out_dtype: x's type (the default) or
    float32. act: none, relu, silu, gelu. residual may be out itself."""
    return _t.linear(x, w, bias, act, residual, out, out_dtype, w_t)


def gated_ffn(x, wg, wu, act="silu", out=None):
    """act(x @ wg.T) * (x @ wu.T) for x [m, d], wg and wu [f, d] (rows may be interleaved)."""
    return _t.gated_ffn(x, wg, wu, act, out)


def gated_ffn_backward(x, wg, wu, dh, act="silu"):
    """(dx, dwg, dwu) of gated_ffn for the gradient dh [m, f] of its result.

    The gradients of x @ wg.T and x @ wu.T are held in x's type: in float16 scale dh (all is linear in
    it) so that they stay below 65,504 and above 6e-5."""
    return _t.gated_ffn_backward(x, wg, wu, dh, act)


def prompt_attention(q, k, v, kv_len, scale=None, out=None):
    """Causal attention of the n new tokens q [n, heads, hd] over a cache k, v [kv_heads, S, hd].

    The cache holds kv_len earlier positions and the n new ones (S >= kv_len + n); token i sees
    the positions up to kv_len + i. scale: 1 / sqrt(hd) unless given. v has to be finite at
    all kv_len + n positions; what lies behind them is not read."""
    return _t.prompt_attention(q, k, v, kv_len, scale, out)
