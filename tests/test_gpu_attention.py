"""kd_prompt_attention on the GPU against its definition in 64 bits.

Bound of one output: p_j is computed in fp32 from a score that is off by e_s (a sum of hd exact
products, and the exponential's few 2^-22), so the weights are off by e_s relative, each is then
rounded to the type (half a step t), and the result is rounded to it: |err| <= (2 e_s + t) *
sum_j p_j |v_j| + t |o|, and sum_err of the second product's sum."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import close, half_step, sum_err

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def reference(q, k, v, kv_len, scale):
    n, hq, hd = q.shape
    T, r = kv_len + n, hq // k.shape[0]
    out = torch.empty(n, hq, hd, dtype=torch.float64, device=q.device)
    mag, err = torch.empty_like(out), torch.empty_like(out)
    at = kv_len + torch.arange(n, device=q.device)
    mask = torch.arange(T, device=q.device)[None] <= at[:, None]
    for h in range(hq):
        K, V, Q = k[h // r, :T].double(), v[h // r, :T].double(), q[:, h].double()
        z = scale * (Q @ K.t())
        es = scale * sum_err(hd) * (Q.abs() @ K.abs().t()) + 2.0 ** -21 * (1 + z.abs())
        es = es.masked_fill(~mask, 0).amax(1, keepdim=True)
        p = torch.softmax(z.masked_fill(~mask, float("-inf")), 1)
        out[:, h], mag[:, h] = p @ V, p @ V.abs()
        err[:, h] = es
    return out, mag, err


def check(n, kv_len, hq, hkv, hd, dt=BF, scale=None, spread=1.0, layout="head", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = n + kv_len
    cap = T + 37
    q = (torch.randn(n, hq, hd, generator=g, device="cuda") * spread).to(dt)
    shape = (hkv, cap, hd) if layout == "head" else (cap, hkv, hd)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
    if layout != "head":
        k, v = k.transpose(0, 1), v.transpose(0, 1)
    k[:, T:] = float("nan")  # what the cache holds behind the last position is never used
    v[:, T:] = float("nan")
    out = torch.full((n + 2, hq, hd), 7.0, dtype=dt, device="cuda")
    kd.prompt_attention(q, k, v, kv_len, scale=scale, out=out[:n])
    kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    assert bool((out[n:] == 7.0).all())
    scale = hd ** -0.5 if scale is None else scale
    want, mag, es = reference(q, k, v, kv_len, scale)
    t = half_step(dt)
    # a weight below the type's normal range loses up to half its smallest subnormal, relative to
    # a largest weight of at least 2^-8 (the reference is raised once it lags by 2^8)
    low = torch.finfo(dt).tiny * t * 2 ** 8 * T * v[:, :T].double().abs().max()
    bound = (2 * es + t + sum_err(T)) * mag + low
    close(out[:n], want, bound + t * (want.abs() + bound) + torch.finfo(dt).tiny, "attention %s" % ((n, kv_len, hq, hkv, hd),))
    rel = float((out[:n].double() - want).norm() / want.norm())
    assert rel <= 2 * t + 2 * float(es.max()), rel


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,kv_len,hq,hkv", [
    (1, 0, 1, 1), (1, 1, 2, 1), (1, 127, 4, 2), (1, 128, 4, 2), (1, 129, 16, 8), (1, 4000, 8, 1), (1, 32768, 16, 8), (2, 5, 6, 2),
    (3, 1000, 32, 4), (16, 0, 8, 8), (31, 97, 12, 4), (42, 0, 3, 1), (43, 0, 3, 1), (64, 64, 2, 1), (65, 300, 16, 8), (77, 1001, 4, 2),
    (128, 0, 1, 1), (129, 0, 4, 4), (300, 0, 16, 8), (257, 500, 32, 8), (5, 700, 5, 1), (9, 33, 128, 1)])
def test_sizes(n, kv_len, hq, hkv, hd):
    check(n, kv_len, hq, hkv, hd)


@pytest.mark.parametrize("n,kv_len", [(1, 500), (50, 30), (700, 100)])
def test_fp16(n, kv_len):
    check(n, kv_len, 8, 4, 128, HF)
    check(n, kv_len, 8, 4, 64, HF)


@pytest.mark.parametrize("n,kv_len", [(1, 2000), (90, 300), (1200, 0)])
def test_sharp_scores_raise_the_reference(n, kv_len):
    """Scores of spread 20: the running maximum grows by more than 2^8 many times."""
    check(n, kv_len, 16, 8, 128, spread=20.0)


def test_positions_before_heads_and_scale():
    check(100, 60, 8, 2, 128, scale=0.3, layout="position")
    check(1, 700, 8, 2, 64, scale=0.01, layout="position")


def test_growing_keys_and_equal_keys():
    """Every key larger than the ones before it: the reference moves at every block; equal keys
    give the mean of the values."""
    n, T, hd = 1, 3000, 128
    q = torch.ones(n, 2, hd, device="cuda", dtype=BF)
    k = (torch.arange(T, device="cuda").float()[None, :, None] / 16).expand(1, T, hd).to(BF).contiguous()
    v = torch.randn(1, T, hd, device="cuda").to(BF)
    out = kd.prompt_attention(q, k, v, T - n)
    want, mag, es = reference(q, k, v, T - n, hd ** -0.5)
    close(out, want, (2 * es + 2 * half_step(BF)) * mag + half_step(BF) * want.abs(), "growing")
    k.zero_()
    out = kd.prompt_attention(q, k, v, T - n)
    mean = v.double().mean(1)
    close(out[0, 0], mean[0], half_step(BF) * mean[0].abs() + sum_err(T) * v.double().abs().mean(1)[0], "mean")


def test_long_prompt():
    check(2500, 0, 8, 2, 128)
    check(1111, 2222, 6, 2, 64)
