"""What the prompt operators refuse on the host, without a GPU: sizes whose 32-bit indices would not hold, a
limit of no time."""

import pytest

from persistent_monokernel_sm_b200 import build

build.build()
import persistent_monokernel_sm_b200 as kd  # noqa: E402

P = 1 << 20  # an aligned address that nothing reads
LD = 1 << 31


@pytest.mark.parametrize("m", [1, 2, 300])
@pytest.mark.parametrize("k", [(1 << 31) - 16383, (1 << 31) - 12288, (1 << 31) - 1025, (1 << 31) - 1])
def test_a_k_whose_steps_pass_32_bits(m, k):
    """The kernel for few tokens steps over k by up to 12,288 in 32 bits: above 2^31 less that, a step past the
    end would wrap to a place before the row."""
    a = kd.kd_linear_args(dtype=0, out_dtype=0, act=0, w_transposed=0, m=m, n=4, k=k, x=P, ld_x=LD, w=P, ld_w=LD, out=P, ld_out=8)
    assert kd.load_library().kd_linear(bytes(a), None) == -1
    g = kd.kd_gated_args(dtype=0, act=2, m=m, d=k, f=4, x=P, ld_x=LD, wg=P, ld_wg=LD, wu=P, ld_wu=LD)
    assert kd.load_library().kd_gated_ffn(bytes(g), P, 8, None) == -1
    assert b"range" in kd.load_library().kd_op_error()


def test_a_limit_of_no_time():
    lib = kd.load_library()
    assert lib.kd_op_set_timeout(0) == -1 and lib.kd_op_set_timeout(-5) == -1
    assert lib.kd_op_set_timeout((1 << 63) - 1) == 0 and lib.kd_op_set_timeout(2_000_000_000) == 0
