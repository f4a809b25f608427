"""The range of fp16 in the gated block's gradients: dg and du are held in it between the products."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import half_step, rows

pytestmark = pytest.mark.gpu
HF = torch.float16


@pytest.mark.parametrize("act", ["silu", "none"])
def test_fp16_gradients_near_the_ends_of_the_range(act):
    """dg and du are held in fp16: a dh that takes them to a few thousand or to 1e-4 keeps the tolerances, one
    that takes them past 65,504 gives infinities or NaN and no finite wrong value; dh scaled by a power of two
    gives the gradients scaled."""
    g = torch.Generator(device="cuda").manual_seed(8)
    m, d, f = 64, 128, 96
    x = rows(g, m, d, 1.0, HF, "cuda")
    wg, wu = rows(g, f, d, 0.05, HF, "cuda"), rows(g, f, d, 0.05, HF, "cuda")
    dh = rows(g, m, f, 1.0, HF, "cuda", pad=1)
    mid = kd.gated_ffn_backward(x, wg, wu, dh, act=act)
    # Scaled by a power of two, values round alike, except those below the normal range on either side: there
    # a term (2 f of them in dx, m in the others) is off by up to half a smallest subnormal, tiny * t, of its own
    # scale, times a weight (an input). A result may then round to the other neighbour: 2 t of it, or half a
    # smallest subnormal on each side where it is below the normal range itself.
    t, tiny = half_step(HF), torch.finfo(HF).tiny
    wide = 2 * f * float(torch.maximum(wg.abs().max(), wu.abs().max())), m * float(x.abs().max())
    for scale in (2.0 ** 7, 2.0 ** -7):
        for i, (a, b) in enumerate(zip(kd.gated_ffn_backward(x, wg, wu, dh * scale, act=act), mid)):
            a, b = a.double() / scale, b.double()
            slack = tiny * t * (1 + 1 / scale) * ((wide[0] if i == 0 else wide[1]) + 1)
            assert bool(((a - b).abs() <= slack + 2 * t * (b.abs() + slack)).all()), (scale, i)
    big = kd.gated_ffn_backward(x, wg, wu, dh * 2.0 ** 13 * 1.9, act=act)
    plain = [b.double() * 2.0 ** 13 * 1.9 for b in mid]
    for a, b in zip(big, plain):
        fine = torch.isfinite(a)
        assert bool(((a.double() - b).abs() <= 6 * t * b.abs().max())[fine].all())
