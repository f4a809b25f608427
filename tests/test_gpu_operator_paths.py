"""The ways a product is cut, each by sizes that take it on a B200 (148 SMs; clusters of 2, 4, 8 CTAs: 74,
33, 15 at once): pairs of CTAs with tiles of 192 and 256 columns, single CTAs with the widths between, a
reduction split over a cluster. Against 64 bits, and as they are used: repeated, captured, on two streams,
in place. Gradients against differences, with a bound that a wrong term does not pass."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import act64, half_step, rows
from tests.test_gpu_gated import check_backward, check_forward
from tests.test_gpu_linear import check

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("m,n,k", [(1000, 1000, 520), (1344, 1000, 256), (1920, 1000, 1032), (1000, 2048, 2048), (700, 9000, 300),
                                   (1344, 2048, 1032), (1501, 2049, 1032), (2048, 2048, 2048)])
def test_linear_widths(m, n, k):
    """Tiles of 96, 96, 160, 192 (pairs), 192 (pairs), 224, 256 (pairs), 256 (pairs) columns."""
    check(m, n, k, bias=True, act="silu")
    check(m, n, k, HF, out=F32, res=True)
    check(m, n, k, w_t=True, out=F32)


@pytest.mark.parametrize("m,n,k", [(161, 1000, 2048), (257, 1000, 2048), (5, 512, 4096), (40, 128, 9000)])
def test_linear_splits(m, n, k):
    check(m, n, k, bias=True, act="gelu", res=True)
    check(m, n, k, w_t=True, out=F32, res=True)


@pytest.mark.parametrize("m,d,f", [(1500, 512, 1000), (190, 512, 8192), (448, 1024, 3000), (1500, 1024, 1000), (2048, 512, 4096)])
def test_gated_widths(m, d, f):
    """Tiles of 192 (pairs), 192 (pairs), 224, 256 (pairs), 256 (pairs) columns."""
    check_forward(m, d, f, act="gelu")
    check_backward(m, d, f, HF)


def pair_calls(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(x=rows(g, 2048, 2048, 1.0, BF, "cuda"), w=rows(g, 2048, 2048, 0.02, BF, "cuda"),
             r=rows(g, 2048, 2048, 1.0, F32, "cuda"), xg=rows(g, 1500, 512, 1.0, BF, "cuda"), wg=rows(g, 4096, 512, 0.05, BF, "cuda"),
             wu=rows(g, 4096, 512, 0.05, BF, "cuda"), dh=rows(g, 1500, 4096, 0.1, BF, "cuda"), xs=rows(g, 40, 2048, 1.0, BF, "cuda"))
    run = {
        "linear": lambda s: [kd.linear(s["x"], s["w"], act="gelu")],
        "linear_f32": lambda s: [kd.linear(s["x"], s["w"], residual=s["r"], out_dtype=F32, w_t=True)],
        "gated": lambda s: [kd.gated_ffn(s["xg"], s["wg"], s["wu"])],
        "gated_bwd": lambda s: list(kd.gated_ffn_backward(s["xg"], s["wg"], s["wu"], s["dh"])),
        "split": lambda s: [kd.linear(s["xs"], s["w"], out_dtype=F32, w_t=True)],
    }
    return s, run


NAMES = ["linear", "linear_f32", "gated", "gated_bwd", "split"]


@pytest.mark.parametrize("name", NAMES)
def test_repeated_and_captured(name):
    s, run = pair_calls(0)
    first = run[name](s)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run[name](s)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run[name](s)
    other, _ = pair_calls(1)
    for k in s:
        s[k].copy_(other[k])
    want = run[name](s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_two_streams_at_once():
    states = [pair_calls(i) for i in range(2)]
    want = [{n: run[n](s) for n in NAMES} for s, run in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for n in NAMES:
            for i, (s, run) in enumerate(states):
                with torch.cuda.stream(streams[i]):
                    got[i].append((n, run[n](s)))
    torch.cuda.synchronize()
    for i in range(2):
        for n, outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i][n], outs)), n
        kd.kd_op_sync(streams[i].cuda_stream)


def test_residual_in_place():
    s, run = pair_calls(2)
    want, = run["linear_f32"](s)
    kd.linear(s["x"], s["w"], residual=s["r"], out=s["r"], w_t=True)
    assert torch.equal(s["r"], want)


@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_gradients_against_differences(act, dt):
    """A gradient's rounding errors e have |e| <= 2 t |gradient| (rounding of dg, du and of the result); a
    direction v that is drawn apart from them makes e.v normal with that deviation, so that six of them, 12 t
    |gradient| (0.05 of it in bf16), are not passed by chance. Central differences of sum(dh * h) in 64 bits: 1e-6."""
    g = torch.Generator(device="cuda").manual_seed(6)
    m, d, f = 33, 72, 90
    x, wg, wu = rows(g, m, d, 1.0, dt, "cuda"), rows(g, f, d, 0.1, dt, "cuda"), rows(g, f, d, 0.1, dt, "cuda")
    dh = rows(g, m, f, 1.0, dt, "cuda", pad=1)
    grads = kd.gated_ffn_backward(x, wg, wu, dh, act=act)
    base = [t.double() for t in (x, wg, wu)]

    def loss(p):
        return (dh.double() * act64(act, p[0] @ p[1].t()) * (p[0] @ p[2].t())).sum()

    for i in range(3):
        size = float(grads[i].double().norm())
        for _ in range(8):
            v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
            eps = 1e-5
            up, down = [list(base) for _ in range(2)]
            up[i], down[i] = base[i] + eps * v, base[i] - eps * v
            want = float((loss(up) - loss(down)) / (2 * eps))
            got = float((grads[i].double() * v).sum())
            assert abs(got - want) <= 12 * half_step(dt) * size + 1e-6 * abs(want), (act, i)
