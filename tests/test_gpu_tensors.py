"""The prompt operators as functions of torch tensors: what they refuse or mark because a gradient would be
lost without a word."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def z(*s):
    return torch.zeros(s, dtype=BF, device="cuda")


def calls(x, w):
    """Each operator with x or w in every place that takes an input."""
    k = z(2, 16, 64)
    q = x.repeat(1, 16).view(2, 4, 64)
    return [lambda: kd.linear(x, w), lambda: kd.linear(z(2, 16), z(16, 16), residual=x), lambda: kd.linear(z(2, 16), z(16, 16), bias=w[0]),
            lambda: kd.gated_ffn(x, w, w), lambda: kd.gated_ffn(z(2, 16), w, z(16, 16)), lambda: kd.gated_ffn(z(2, 16), z(16, 16), w),
            lambda: kd.gated_ffn_backward(x, w, w, z(2, 16)), lambda: kd.gated_ffn_backward(z(2, 16), z(16, 16), z(16, 16), x),
            lambda: kd.prompt_attention(q, k, k, 3)]


def test_inputs_that_require_grad():
    """No graph is recorded: such a call is refused where gradients are, and runs where they are not."""
    x, w = z(2, 16).requires_grad_(), z(16, 16).requires_grad_()
    for call in calls(x, w):
        with pytest.raises(kd.KdError) as e:
            call()
        assert e.value.code == -1 and "no_grad" in str(e.value)
    with torch.no_grad():
        for call in calls(x, w):
            call()
    for call in calls(x.detach(), w.detach()):
        call()
    k = z(2, 16, 64).requires_grad_()
    for a in ((z(2, 4, 64), k, z(2, 16, 64)), (z(2, 4, 64), z(2, 16, 64), k)):
        with pytest.raises(kd.KdError):
            kd.prompt_attention(*a, 3)


def test_an_output_that_requires_grad():
    out = z(2, 16).requires_grad_()
    with pytest.raises(kd.KdError):
        kd.linear(z(2, 16), z(16, 16), out=out)
    with pytest.raises(kd.KdError):
        kd.gated_ffn(z(2, 16), z(16, 16), z(16, 16), out=out)
    with pytest.raises(kd.KdError):
        kd.prompt_attention(z(2, 4, 64), z(2, 16, 64), z(2, 16, 64), 3, out=z(2, 4, 64).requires_grad_())


def test_a_written_output_counts_as_changed():
    """torch then refuses a backward pass that needs the value which was written over."""
    for write in (lambda o: kd.linear(z(2, 16), z(16, 16), out=o), lambda o: kd.gated_ffn(z(2, 16), z(16, 16), z(16, 16), out=o),
                  lambda o: kd.linear(z(2, 16), z(16, 16), residual=o, out=o)):
        o = z(2, 16)
        p = torch.ones(2, 16, dtype=BF, device="cuda", requires_grad=True)
        y = (p * o).sum()
        before = o._version
        write(o)
        assert o._version == before + 1
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    o = z(2, 4, 64)
    kd.prompt_attention(z(2, 4, 64), z(2, 16, 64), z(2, 16, 64), 3, out=o)
    assert o._version == 1
    with torch.inference_mode():
        kd.linear(z(2, 16), z(16, 16), out=z(2, 16))


def test_arguments_that_are_no_numbers():
    with pytest.raises((RuntimeError, ValueError)):
        kd.linear(z(2, 16), z(16, 16), w_t=torch.ones(2))  # of no one truth value
    for kv in (1 << 62, (1 << 63) - 1):
        with pytest.raises(kd.KdError):
            kd.prompt_attention(z(2, 4, 64), z(2, 16, 64), z(2, 16, 64), kv)
