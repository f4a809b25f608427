"""Plain 64-bit forms of the prompt operators, and the rounding bounds their tests count with.

A result of fp32 sums rounded once to the output type t is off by at most half a step of t,
eps(t)/2 relative, plus the error of the sums. Products of two 16-bit values are exact in fp32;
a sum of K of them in any order is off by at most K * 2^-24 * sum|terms| in the worst case and
by about sqrt(K) * 2^-24 of it in practice: the tests allow sum_err(K) = (8 + sqrt(K)) * 2^-23
of the sum of the terms' magnitudes (a tensor core may truncate where fp32 rounds: 2^-23)."""

import math

import torch



def half_step(t):
    return torch.finfo(t).eps / 2


def sum_err(k):
    return (8 + math.sqrt(k)) * 2.0 ** -23


def act64(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def slope64(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def close(got, want, bound, what=""):
    """|got - want| <= bound elementwise (64-bit tensors)."""
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, d / bound.clamp_min(1e-300), torch.zeros_like(d)).flatten()))
        raise AssertionError("%s: %d of %d off; worst at %d: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]),
            float(bound.flatten()[i])))


def rows(g, r, c, scale, dt, device, pad=8, extra=0):
    """[r][c] with rows that start on a multiple of `pad` elements (+ extra); the padding is NaN."""
    ld = -(-c // pad) * pad + extra
    t = torch.full((r, ld), float("nan"), dtype=dt, device=device)
    t[:, :c] = (torch.randn(r, c, generator=g, device=device) * scale).to(dt)
    return t[:, :c]
