"""Operators whose device-side waits run out of their limit: the kernels end early, without a trap or a hang,
kd_op_sync reports it once, and the next calls are as before.

With a limit of 1 ns the first wait that does not succeed at once gives up: that of the issuer for the first
tile, whose copies have just been started, while the producer may have started all of its own."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import rows

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def limit():
    yield kd.kd_op_set_timeout
    kd.kd_op_set_timeout(2_000_000_000)


def calls():
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = rows(g, 40, 1000, 1.0, BF, "cuda"), rows(g, 300, 1000, 0.05, BF, "cuda")
    xl, wl = rows(g, 2048, 2048, 1.0, BF, "cuda"), rows(g, 2048, 2048, 0.05, BF, "cuda")
    xg, wg, wu = rows(g, 1500, 512, 1.0, BF, "cuda"), rows(g, 4096, 512, 0.05, BF, "cuda"), rows(g, 4096, 512, 0.05, BF, "cuda")
    dh, dhl = rows(g, 40, 300, 0.1, BF, "cuda", pad=1), rows(g, 1500, 4096, 0.1, BF, "cuda")
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((3, 8, 128), (4, 3000, 128), (4, 3000, 128)))
    ql = torch.randn(2500, 8, 128, generator=g, device="cuda").to(BF)
    qs, ks = torch.randn(1500, 16, 64, generator=g, device="cuda").to(BF), torch.randn(8, 1600, 64, generator=g, device="cuda").to(BF)
    return {
        "linear": lambda: [kd.linear(x, w, act="gelu")],                                       # single CTAs
        "linear_short": lambda: [kd.linear(x[:, :64], w[:, :64])],                             # one k-block
        "linear_split": lambda: [kd.linear(xl[:40], wl, out_dtype=F32, w_t=True)],             # a cluster's split
        "linear_pairs": lambda: [kd.linear(xl, wl), kd.linear(xl, wl, out_dtype=F32, w_t=True)],
        "gated": lambda: [kd.gated_ffn(x, w, w)],
        "gated_pairs": lambda: [kd.gated_ffn(xg, wg, wu)],
        "backward": lambda: list(kd.gated_ffn_backward(x, w, w, dh)),
        "backward_pairs": lambda: list(kd.gated_ffn_backward(xg, wg, wu, dhl)),
        "attention_split": lambda: [kd.prompt_attention(q, k, v, 2900)],
        "attention_one_block": lambda: [kd.prompt_attention(q, k, v, 0)],
        "attention": lambda: [kd.prompt_attention(ql, k, v, 400)],                             # whole tiles
        "attention_64": lambda: [kd.prompt_attention(qs, ks, ks, 100)],
    }


NAMES = ["linear", "linear_short", "linear_split", "linear_pairs", "gated", "gated_pairs", "backward", "backward_pairs",
         "attention_split", "attention_one_block", "attention", "attention_64"]


def status():
    try:
        kd.kd_op_sync(torch.cuda.current_stream().cuda_stream)
    except kd.KdError as e:
        return e.code
    return 0


@pytest.mark.parametrize("name", NAMES)
def test_a_wait_that_runs_out(name, limit):
    run = calls()[name]
    want = run()
    assert status() == 0
    for _ in range(3):
        limit(1)
        run()
        limit(2_000_000_000)
        assert status() == -6
        assert status() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
        assert status() == 0


def test_the_limit_belongs_to_the_thread_and_to_the_call(limit):
    import concurrent.futures
    run = calls()["linear"]
    limit(1)
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        want = pool.submit(run).result()
    assert status() == 0
    graph = torch.cuda.CUDAGraph()
    limit(2_000_000_000)
    with torch.cuda.graph(graph):
        got = run()
    limit(1)
    graph.replay()  # keeps the limit that it was captured with
    assert status() == 0 and torch.equal(got[0], want[0])


@pytest.mark.parametrize("name", [n for n in NAMES if "pairs" not in n])
def test_a_short_limit_that_is_not_exceeded(name, limit):
    """0.4 ms, where no wait of these calls takes a tenth of it."""
    run = calls()[name]
    want = run()
    torch.cuda.synchronize()
    limit(400_000)
    got = run()
    assert status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_limit_of_no_time_is_refused():
    for ns in (0, -1):
        with pytest.raises(kd.KdError) as e:
            kd.kd_op_set_timeout(ns)
        assert e.value.code == -1
