"""Scores that are not finite, through every way the attention cuts its work: one tile with two
streams, tiles split over CTAs and joined, whole tiles. A NaN that a row sees is a NaN in its
result wherever it lies; a row that does not see it keeps its bits."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import half_step, sum_err
from tests.test_gpu_attention import reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# (n, kv_len, heads, kv heads, head dim, first and last poisoned position): the only position of the
# last block (of a CTA, of a stream), a whole block, a position among others
CASES = [(1, 128, 16, 8, 128, 128, 128), (1, 1024, 16, 8, 128, 1024, 1024), (1, 128, 160, 80, 128, 128, 128),
         (1, 128, 160, 80, 64, 0, 127), (1, 1000, 16, 8, 128, 0, 127), (1, 4000, 16, 8, 128, 256, 383),
         (1, 32768, 16, 8, 128, 5000, 5000), (77, 1001, 4, 2, 64, 256, 383), (3, 126, 4, 2, 64, 128, 128),
         (300, 0, 4, 2, 64, 200, 200), (300, 0, 16, 8, 128, 128, 255), (2000, 0, 32, 8, 128, 1024, 1151)]


def make(n, kv_len, hq, hkv, hd, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = n + kv_len
    return [torch.randn(s, generator=g, device="cuda").to(BF) for s in ((n, hq, hd), (hkv, T, hd), (hkv, T, hd))]


@pytest.mark.parametrize("n,kv_len,hq,hkv,hd,lo,hi", CASES)
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_key_that_is_not_finite(n, kv_len, hq, hkv, hd, lo, hi, what):
    """A key of NaN, or one whose score is +infinity (infinity less infinity in the softmax), in the last
    kv head: NaN in that head's rows which see it, the same bits everywhere else."""
    q, k, v = make(n, kv_len, hq, hkv, hd)
    if what == "inf":
        q = q.abs() + 0.01
    clean = kd.prompt_attention(q, k, v, kv_len)
    k[hkv - 1, lo:hi + 1] = float(what)
    got = kd.prompt_attention(q, k, v, kv_len)
    sees = kv_len + torch.arange(n, device="cuda") >= lo
    poisoned = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    poisoned[:, (hkv - 1) * (hq // hkv):] = sees[:, None]
    assert bool(torch.isnan(got[poisoned]).all())
    assert torch.equal(got[~poisoned], clean[~poisoned])


@pytest.mark.parametrize("n,kv_len,hq,hkv,hd,lo,hi", CASES)
def test_scores_of_minus_infinity_have_no_weight(n, kv_len, hq, hkv, hd, lo, hi):
    """As if the positions were not there; where a row sees nothing else its result is NaN (0 / 0)."""
    q, k, v = make(n, kv_len, hq, hkv, hd, 1)
    q = q.abs() + 0.01
    k[:, lo:hi + 1] = -float("inf")
    got = kd.prompt_attention(q, k, v, kv_len)
    there = torch.ones(n + kv_len, dtype=torch.bool, device="cuda")
    there[lo:hi + 1] = False
    rows = kv_len + torch.arange(n, device="cuda")
    empty = torch.cumsum(there, 0)[rows] == 0
    assert bool(torch.isnan(got[empty]).all())
    # row by row over what is left: a sample of rows, each as the last token behind the remaining cache
    keep = [i for i in sorted({0, n // 2, n - 1}) if not bool(empty[i])]
    for i in keep:
        see = there[:kv_len + i + 1]
        kk, vv = k[:, :kv_len + i + 1][:, see], v[:, :kv_len + i + 1][:, see]
        want, mag, es = reference(q[i:i + 1], kk, vv, kk.shape[1] - 1, hd ** -0.5)
        t = half_step(BF)
        # weights that fall below the type's normal range: as in the attention's own tests
        low = torch.finfo(BF).tiny * t * 2 ** 8 * kk.shape[1] * vv.double().abs().max()
        bound = (2 * es + t + sum_err(kk.shape[1])) * mag + low
        assert bool(((got[i:i + 1].double() - want).abs() <= bound + t * (want.abs() + bound) + torch.finfo(BF).tiny).all())
