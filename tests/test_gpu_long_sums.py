"""Long sums rounded to 16 bits. All terms have one sign, so that an accumulator which is truncated towards
zero at every step is off by the whole of it: 6.5e-3 measured over the 2^20 products of a CTA here (2^23 split
eight ways), where the half steps are 4.9e-4 (fp16) and 3.9e-3 (bf16). The bound is that of the other tests: a
rounding of the result, and sum_err of fp32 sums."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import close, half_step, sum_err

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
K = 1 << 23


def positive(g, shape, lo, dt):
    """Uniform in [lo, 2 lo)."""
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32).add_(1).mul_(lo).to(dt)


def product64(a, b):
    """a [m][K] @ b [n][K]^T in 64 bits, a piece of K at a time."""
    out = 0
    for i in range(0, K, 1 << 18):
        out = out + a[:, i:i + (1 << 18)].double() @ b[:, i:i + (1 << 18)].double().t()
    return out


def held(got, want, dt):
    bound = sum_err(K) * want
    close(got, want, bound + half_step(dt) * (want + bound), "long sum")


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("w_t", [False, True])
def test_linear(dt, w_t):
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = positive(g, (8, K), 0.5, dt), positive(g, (40, K), 0.004, dt)
    want = product64(x, w)
    got = kd.linear(x, w.t().contiguous() if w_t else w, w_t=w_t)
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    held(got, want, dt)


@pytest.mark.parametrize("dt", [HF, BF])
def test_weight_gradients_over_many_tokens(dt):
    """wg and wu pick x's first column, which is 1, and there is no activation: dg = du = dh exactly, and both
    gradients are dh^T x."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dh = positive(g, (K, 16), 0.5, dt), positive(g, (K, 8), 0.004, dt)
    x[:, 0] = 1
    w = torch.zeros(8, 16, dtype=dt, device="cuda")
    w[:, 0] = 1
    want = product64(dh.t().contiguous(), x.t().contiguous())
    _, dwg, dwu = kd.gated_ffn_backward(x, w, w, dh, act="none")
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    held(dwg, want, dt)
    held(dwu, want, dt)
