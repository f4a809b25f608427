"""The prompt operators as the first CUDA call of a host thread, which has no context current yet: an
autograd worker, a server's pool."""

import concurrent.futures

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.test_gpu_operators import NAMES, calls

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        return pool.submit(f).result()


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_thread(name):
    s, run = calls()
    want = run[name](s)
    got = in_a_new_thread(lambda: run[name](s))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_from_a_backward_pass():
    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wg, wu):
            ctx.save_for_backward(x, wg, wu)
            return kd.gated_ffn(x, wg, wu)

        @staticmethod
        def backward(ctx, dh):
            return kd.gated_ffn_backward(*ctx.saved_tensors, dh)

    g = torch.Generator(device="cuda").manual_seed(0)
    x, wg, wu = [(torch.randn(s, generator=g, device="cuda") * 0.3).to(torch.bfloat16).requires_grad_() for s in ((9, 64), (40, 64), (40, 64))]
    dh = torch.randn(9, 40, generator=g, device="cuda").to(torch.bfloat16)
    Block.apply(x, wg, wu).backward(dh)
    want = kd.gated_ffn_backward(x.detach(), wg.detach(), wu.detach(), dh)
    for p, w in zip((x, wg, wu), want):
        assert torch.equal(p.grad, w)


def test_several_threads_at_once():
    states = [calls(i) for i in range(4)]
    want = [{n: run[n](s) for n in NAMES} for s, run in states]
    torch.cuda.synchronize()

    def work(i):
        s, run = states[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [(n, run[n](s)) for _ in range(10) for n in NAMES]
            torch.cuda.current_stream().synchronize()
            kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
        return all(torch.equal(a, b) for n, outs in got for a, b in zip(want[i][n], outs))

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))
