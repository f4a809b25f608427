"""kd_gated_ffn and its backward pass on the GPU against their definitions in 64 bits."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import act64, close, half_step, rows, slope64, sum_err

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def make(m, d, f, dt, extra=0, seed=0, interleaved=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = rows(g, m, d, 1.0, dt, "cuda", extra=extra)
    if interleaved:
        w = rows(g, 2 * f, d, 0.05, dt, "cuda", extra=extra)
        wg, wu = w[0::2], w[1::2]
    else:
        wg, wu = rows(g, f, d, 0.05, dt, "cuda", extra=extra), rows(g, f, d, 0.05, dt, "cuda", extra=extra)
    dh = rows(g, m, f, 0.1, dt, "cuda", pad=1, extra=extra)
    return x, wg, wu, dh


def terms(x, wg, wu):
    X, G, U = x.double(), wg.double(), wu.double()
    e = sum_err(x.shape[1])
    g, u = X @ G.t(), X @ U.t()
    return g, u, e * (X.abs() @ G.abs().t()), e * (X.abs() @ U.abs().t())


def check_forward(m, d, f, dt=BF, act="silu", **kw):
    x, wg, wu, _ = make(m, d, f, dt, **kw)
    buf = torch.full((m, f + 3), 7.0, dtype=dt, device="cuda")
    got = kd.gated_ffn(x, wg, wu, act=act, out=buf[:, :f])
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    assert bool((buf[:, f:] == 7.0).all())
    g, u, eg, eu = terms(x, wg, wu)
    a = act64(act, g)
    ea = 1.13 * eg + 2.0 ** -21 * (g.abs() + 1)
    h = a * u
    bound = ea * (u.abs() + eu) + a.abs() * eu
    close(got, h, bound + half_step(dt) * (h.abs() + bound) + torch.finfo(dt).tiny, "gated %s" % ((m, d, f),))


def check_backward(m, d, f, dt=BF, act="silu", **kw):
    x, wg, wu, dh = make(m, d, f, dt, **kw)
    dx, dwg, dwu = kd.gated_ffn_backward(x, wg, wu, dh, act=act)
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    g, u, eg, eu = terms(x, wg, wu)
    X, D = x.double(), dh.double()
    a, s = act64(act, g), slope64(act, g)
    dg, du = D * u * s, D * a
    # each is computed in fp32 from g and u that are off by eg and eu (|act''| <= 1 for silu and
    # gelu; relu's slope jumps where g is within eg of 0) and rounded once to dt
    es = torch.where(g.abs() <= eg, 1.0, 0.0) if act == "relu" else eg + 2.0 ** -20 * (g.abs() + 1)
    # half a smallest subnormal: what rounding may lose of a value below the normal range
    t = half_step(dt)
    sub = torch.finfo(dt).tiny * t
    bg = D.abs() * (u.abs() * es + (s.abs() + es) * eu) + t * dg.abs() * 1.01 + sub
    bu = D.abs() * (1.13 * eg + 2.0 ** -21 * (g.abs() + 1)) + t * du.abs() * 1.01 + sub
    G, U = wg.double(), wu.double()
    for name, got, want, err, mag, k in (
            ("dx", dx, dg @ G + du @ U, bg @ G.abs() + bu @ U.abs(), dg.abs() @ G.abs() + du.abs() @ U.abs(), 2 * f),
            ("dwg", dwg, dg.t() @ X, bg.t() @ X.abs(), dg.abs().t() @ X.abs(), m),
            ("dwu", dwu, du.t() @ X, bu.t() @ X.abs(), du.abs().t() @ X.abs(), m)):
        bound = err + sum_err(k) * (mag + err)
        close(got, want, bound + t * (want.abs() + bound) + torch.finfo(dt).tiny, "%s %s" % (name, (m, d, f)))
        # the bound above lets every rounding err the same way; they do not: over the whole
        # output the error is that of roundings of random sign, a few times t
        rel = float((got.double() - want).norm() / want.norm().clamp_min(1e-300))
        assert rel <= 2 * t, (name, rel)


SIZES = [(1, 64, 64), (1, 8, 1), (1, 1536, 500), (2, 72, 65), (3, 136, 63), (15, 64, 200), (17, 256, 129), (64, 128, 64), (65, 520, 301),
         (128, 256, 1001), (200, 64, 33), (257, 256, 1001), (300, 1000, 700)]


@pytest.mark.parametrize("m,d,f", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_forward_sizes(m, d, f, dt):
    check_forward(m, d, f, dt)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_forward_activations_strides_and_interleaved_rows(act):
    check_forward(70, 200, 150, act=act, extra=16)
    check_forward(5, 200, 150, act=act, interleaved=True)


@pytest.mark.parametrize("m,d,f", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_backward_sizes(m, d, f, dt):
    check_backward(m, d, f, dt)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_backward_activations(act):
    check_backward(96, 128, 300, act=act, extra=8)


def test_many_tiles():
    check_forward(1500, 512, 3000)
    check_backward(1500, 512, 3000)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("d,f", [(8, 1), (9, 7), (515, 100), (256, 3000), (9000, 130)])
def test_few_tokens(m, d, f):
    check_forward(m, d, f, act="gelu")
    check_forward(m, d, f, HF, extra=8)
    check_forward(m, d, f, interleaved=True)
