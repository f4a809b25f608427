"""kd_linear on the GPU against its definition in 64 bits."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import act64, close, half_step, rows, sum_err

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def check(m, n, k, dt=BF, out=None, w_t=False, bias=False, act="none", res=False, extra=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = out or dt
    x = rows(g, m, k, 1.0, dt, "cuda", extra=extra)
    w = rows(g, k, n, 0.05, dt, "cuda", extra=extra) if w_t else rows(g, n, k, 0.05, dt, "cuda", extra=extra)
    b = torch.randn(n, generator=g, device="cuda").to(dt) if bias else None
    r = rows(g, m, n, 1.0, out, "cuda", pad=1, extra=extra) if res else None
    buf = torch.full((m, n + 5), 7.0, dtype=out, device="cuda")
    got = kd.linear(x, w, bias=b, act=act, residual=r, out=buf[:, :n], w_t=w_t)
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    assert bool((buf[:, n:] == 7.0).all()), "wrote behind its rows"
    X, W = x.double(), (w.t() if w_t else w).double()
    z = X @ W.t()
    mag = X.abs() @ W.abs().t()
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    y = act64(act, z)
    # |act'| <= 1.13 for every activation here; exp and erf are good to a few 2^-23 of |z| + 1
    bound = 1.13 * sum_err(k) * mag + 2.0 ** -21 * (z.abs() + (act != "none"))
    if res:
        y = y + r.double()
        bound = bound + 2.0 ** -23 * y.abs()
    close(got, y, bound + half_step(out) * (y.abs() + bound) + torch.finfo(out).tiny, "linear %s" % ((m, n, k),))


@pytest.mark.parametrize("m,n,k", [(1, 128, 64), (1, 1, 1), (1, 2, 3), (2, 127, 65), (3, 129, 63), (16, 256, 128), (17, 300, 200),
                                   (33, 64, 1000), (64, 513, 72), (65, 1000, 320), (128, 128, 128),
                                   (129, 255, 777), (255, 1536, 512), (257, 2048, 264), (300, 96, 4096), (1, 5000, 1536),
                                   (1000, 1000, 1000), (5, 20000, 136)])
def test_sizes(m, n, k):
    check(m, n, k)
    check(m, n, k, w_t=True, out=F32, res=True, bias=True)


@pytest.mark.parametrize("dt,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m", [1, 40, 300])
def test_types_and_epilogues(dt, out, act, m):
    check(m, 333, 200, dt, out, bias=True, act=act, res=True)
    check(m, 333, 200, dt, out, w_t=True, act=act)


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 2048), (700, 9000, 300), (4096, 260, 1536)])
def test_many_tiles(m, n, k):
    check(m, n, k, bias=True, act="silu", extra=8)
    check(m, n, k, out=F32, w_t=True, res=True)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,k", [(1, 1), (7, 9), (64, 64), (100, 515), (2400, 256), (1000, 1000), (300, 9000), (3, 20000)])
def test_few_tokens(m, n, k):
    """Either side of the rule between the two kernels, a row of weights per warp and shared by several,
    lengths that are no multiple of 8."""
    check(m, n, k, bias=True, act="gelu", res=True)
    check(m, n, k, HF, out=F32, res=True, extra=8)
    check(m, n, k, HF)


@pytest.mark.parametrize("m", [65, 90, 97, 150, 161, 190, 193, 220, 225, 257, 290])
def test_widths_between_the_powers_of_two(m):
    """Token counts that the plan cuts into tiles of 96, 160, 192 or 224 columns."""
    check(m, 19000, 128, bias=True, act="relu")
    check(m, 5000, 1200, out=F32, res=True)
    check(m, 700, 2400, w_t=True, out=F32)
