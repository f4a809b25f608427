"""How the prompt operators are used on the GPU: streams, graphs, repeated runs, in-place outputs,
empty inputs, values that are not finite, far offsets, gradients against differences."""

import pytest
import torch

import persistent_monokernel_sm_b200 as kd
from tests.operator_util import act64, half_step, rows

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def calls(seed=0):
    """One call of each operator and kind (whole, split over a cluster, split with a workspace)."""
    g = gen(seed)
    x, w = rows(g, 40, 1000, 1.0, BF, "cuda"), rows(g, 300, 1000, 0.05, BF, "cuda")
    x1, w1 = rows(g, 1, 2048, 1.0, BF, "cuda"), rows(g, 512, 2048, 0.05, BF, "cuda")
    wg, wu = rows(g, 500, 1000, 0.05, BF, "cuda"), rows(g, 500, 1000, 0.05, BF, "cuda")
    dh = rows(g, 40, 500, 0.1, BF, "cuda", pad=1)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((3, 8, 128), (4, 3000, 128), (4, 3000, 128)))
    q2 = torch.randn(500, 8, 128, generator=g, device="cuda").to(BF)
    state = dict(x=x, w=w, x1=x1, w1=w1, wg=wg, wu=wu, dh=dh, q=q, k=k, v=v, q2=q2)
    run = {
        "linear": lambda s: [kd.linear(s["x"], s["w"], act="gelu")],
        "linear_split": lambda s: [kd.linear(s["x1"], s["w1"], out_dtype=F32)],
        "gated": lambda s: [kd.gated_ffn(s["x"], s["wg"], s["wu"])],
        "gated_bwd": lambda s: list(kd.gated_ffn_backward(s["x"], s["wg"], s["wu"], s["dh"])),
        "attention_split": lambda s: [kd.prompt_attention(s["q"], s["k"], s["v"], 2900)],
        "attention": lambda s: [kd.prompt_attention(s["q2"], s["k"], s["v"], 0)],
    }
    return state, run


NAMES = ["linear", "linear_split", "gated", "gated_bwd", "attention_split", "attention"]


@pytest.mark.parametrize("name", NAMES)
def test_runs_do_not_differ(name):
    s, run = calls()
    first = run[name](s)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run[name](s)))


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed_on_new_inputs(name):
    s, run = calls(1)
    run[name](s)  # warm-up: what is looked up once per device
    graphs = []
    for _ in range(2):  # two graphs, each with its own outputs and workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run[name](s)
        graphs.append((g, outs))
    other, _ = calls(2)
    for k in s:
        s[k].copy_(other[k])
    want = [t.clone() for t in run[name](s)]
    for g, _ in graphs:
        g.replay()
    for g, _ in reversed(graphs):
        g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_two_streams_at_once():
    states = [calls(i) for i in range(2)]
    want = [{n: [t.clone() for t in run[n](s)] for n in NAMES} for s, run in states]
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


def test_one_after_the_other_reads_what_was_written():
    """Launches that may overlap the end of the one before: a chain through one buffer."""
    g = gen(3)
    w = rows(g, 256, 256, 1 / 16, BF, "cuda")
    a = rows(g, 5, 256, 1.0, BF, "cuda").contiguous()
    want, x = [], a.clone()
    for _ in range(40):
        x = kd.linear(x, w, residual=x)
        torch.cuda.synchronize()
        x = kd.gated_ffn(x, w, w, act="none")
        torch.cuda.synchronize()
        x = (x.float() / x.float().norm() * 30).to(BF)
        want.append(x.clone())
    x = a.clone()
    buf, buf2 = torch.empty_like(x), torch.empty_like(x)
    for i in range(40):
        kd.linear(x, w, residual=x, out=buf)
        kd.gated_ffn(buf, w, w, act="none", out=buf2)
        x = (buf2.float() / buf2.float().norm() * 30).to(BF)
        assert torch.equal(x, want[i])


@pytest.mark.parametrize("m,n,k,out", [(1, 333, 500, F32), (70, 1000, 640, BF), (300, 512, 1100, F32), (1, 2048, 4096, BF)])
def test_residual_in_place(m, n, k, out):
    g = gen(4)
    x, w = rows(g, m, k, 1.0, BF, "cuda"), rows(g, n, k, 0.05, BF, "cuda")
    r = rows(g, m, n, 1.0, out, "cuda", pad=1)
    want = kd.linear(x, w, residual=r, out_dtype=out)
    kd.linear(x, w, residual=r, out=r)
    assert torch.equal(r, want)


def test_empty_inputs():
    z = lambda *s: torch.empty(s, dtype=BF, device="cuda")  # noqa: E731
    assert kd.linear(z(0, 16), z(8, 16)).shape == (0, 8)
    assert kd.linear(z(3, 16), z(0, 16)).shape == (3, 0)
    assert kd.gated_ffn(z(0, 16), z(8, 16), z(8, 16)).shape == (0, 8)
    dx, dwg, dwu = kd.gated_ffn_backward(z(0, 16), z(8, 16), z(8, 16), z(0, 8))
    assert dx.shape == (0, 16) and not dwg.any() and not dwu.any()
    assert kd.prompt_attention(z(0, 4, 64), z(2, 10, 64), z(2, 10, 64), 5).shape == (0, 4, 64)


def test_refused_tensors():
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    k = z(2, 10, 64)
    for call in (lambda: kd.linear(z(2, 16), z(8, 24)), lambda: kd.linear(z(2, 16), z(8, 16, dt=HF)),
                 lambda: kd.linear(z(2, 16), z(8, 16), act="tanh"), lambda: kd.linear(z(2, 16), z(8, 16), out_dtype=HF),
                 lambda: kd.linear(z(2, 16), z(8, 16), bias=z(7)), lambda: kd.linear(z(2, 16), z(8, 16), residual=z(2, 7)),
                 lambda: kd.linear(z(2, 16, dt=F32), z(8, 16, dt=F32)), lambda: kd.linear(z(16, 2).t(), z(8, 16)),
                 lambda: kd.linear(z(2, 17), z(8, 17)), lambda: kd.linear(z(2, 40)[:, 1:17], z(8, 16)),
                 lambda: kd.linear(z(2, 16), z(8, 16), out=z(2, 9)), lambda: kd.linear(z(2, 16), z(8, 16).cpu()),
                 lambda: kd.gated_ffn(z(2, 16), z(8, 16), z(9, 16)), lambda: kd.gated_ffn_backward(z(2, 16), z(8, 16), z(8, 16), z(2, 7)),
                 lambda: kd.prompt_attention(z(3, 3, 64), k, k, 2), lambda: kd.prompt_attention(z(3, 4, 64), k, k, 8),
                 lambda: kd.prompt_attention(z(3, 4, 64), k, z(2, 10, 128), 2), lambda: kd.prompt_attention(z(3, 4, 96), z(2, 10, 96), z(2, 10, 96), 2),
                 lambda: kd.prompt_attention(z(3, 4, 64), k, k, -1), lambda: kd.prompt_attention(z(3, 4, 64), k, k, 2, scale=0.0)):
        with pytest.raises(kd.KdError) as e:
            call()
        assert e.value.code == -1


def test_values_that_are_not_finite_stay_in_their_rows():
    g = gen(5)
    x, w = rows(g, 50, 256, 1.0, BF, "cuda"), rows(g, 200, 256, 0.05, BF, "cuda")
    clean = kd.linear(x, w, act="silu")
    h = kd.gated_ffn(x, w, w)
    x[7, 3], x[20, 5] = float("nan"), float("inf")
    for got, ref in ((kd.linear(x, w, act="silu"), clean), (kd.gated_ffn(x, w, w), h)):
        keep = [i for i in range(50) if i not in (7, 20)]
        assert torch.equal(got[keep], ref[keep])
        assert bool(torch.isnan(got[7]).all()) and not bool(torch.isfinite(got[20]).all())
    # a key that earlier tokens do not see, and one that is seen by all
    n, hq, hkv, hd = 300, 4, 2, 64
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((n, hq, hd), (hkv, n, hd), (hkv, n, hd)))
    ref = kd.prompt_attention(q, k, v, 0)
    k[:, 200] = float("nan")
    got = kd.prompt_attention(q, k, v, 0)
    assert torch.equal(got[:200], ref[:200]) and bool(torch.isnan(got[200:]).all())
    k[:, 200] = 1.0
    q[33] = float("inf")
    got = kd.prompt_attention(q, k, v, 0)
    assert bool(torch.isnan(got[33]).all())
    assert bool(torch.isfinite(got[:33]).all()) and bool(torch.isfinite(got[34:]).all())


def test_offsets_past_32_bits():
    n, hd = 1 << 24, 128
    k, v = (torch.zeros(2, n + 8, hd, dtype=BF, device="cuda") for _ in range(2))  # 2^31 elements to head 1
    v[1, n // 2:] = 1.0
    out = kd.prompt_attention(torch.ones(1, 2, hd, dtype=BF, device="cuda"), k, v, n - 1)
    # every key is equal: the mean of the values, exactly half of which are 1; sums of 2^24 equal weights
    # in fp32 by 128 and joined from few parts are exact
    assert bool((out[0, 0] == 0).all()) and bool((out[0, 1].float() - 0.5).abs().max() <= 0.5 * half_step(BF))
    del k, v
    m, cols = 17000, 128256  # 2^31 outputs and more
    x, w = torch.ones(m, 64, dtype=BF, device="cuda"), torch.zeros(cols, 64, dtype=BF, device="cuda")
    w[:, 0] = (torch.arange(cols, device="cuda") % 251).to(BF)
    y = kd.linear(x, w)
    for i in (0, 1, m // 2, m - 1):
        assert torch.equal(y[i], w[:, 0])


def test_gradients_one_by_one():
    """A NULL output is skipped; the others are what the whole call gives."""
    g = gen(7)
    m, d, f = 70, 128, 200
    x, wg, wu = rows(g, m, d, 1.0, BF, "cuda"), rows(g, f, d, 0.1, BF, "cuda"), rows(g, f, d, 0.1, BF, "cuda")
    dh = rows(g, m, f, 1.0, BF, "cuda", pad=1)
    want = kd.gated_ffn_backward(x, wg, wu, dh)
    args = kd.kd_gated_args(0, 2, m, d, f, x.data_ptr(), x.stride(0), wg.data_ptr(), wg.stride(0), wu.data_ptr(), wu.stride(0))
    n = kd.kd_gated_ffn_backward_workspace(m, f)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
    stream = torch.cuda.current_stream().cuda_stream
    for mask in range(8):
        out = [torch.full((r, d + 8), 7.0, dtype=BF, device="cuda") for r in (m, f, f)]
        p = [o.data_ptr() if mask >> i & 1 else None for i, o in enumerate(out)]
        kd.kd_gated_ffn_backward(args, dh.data_ptr(), f, p[0], d + 8, p[1], d + 8, p[2], d + 8, ws.data_ptr(), n, stream)
        for i in range(3):
            assert torch.equal(out[i][:, :d], want[i]) if mask >> i & 1 else bool((out[i] == 7.0).all())
            assert bool((out[i][:, d:] == 7.0).all())


FIRST_CALL = """
import torch
import persistent_monokernel_sm_b200 as kd
torch.cuda.init()
z = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
x, x1, w, dh, q, k = z(40, 512), z(1, 512), z(64, 512), z(40, 64), z(2, 4, 64), z(2, 2000, 64)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = [kd.linear(x, w), kd.linear(x1, w), kd.gated_ffn(x, w, w), *kd.gated_ffn_backward(x, w, w, dh), kd.prompt_attention(q, k, k, 1990)]
g.replay()
torch.cuda.synchronize()
assert float(outs[0][0, 0]) == 512 and float(outs[1][0, 0]) == 512 and float(outs[-1][0, 0, 0]) == 1
print("captured")
"""


def test_the_first_call_may_be_a_captured_one():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_gradients_against_differences():
    """The gradients' projection on a direction against central differences of sum(dh * h) in 64 bits.
    The kernels' gradients are within 2 half-steps of theirs (rounding of dg, du and the result), so a
    projection is within 2 t |gradient| |direction|; the differences' own error is of order eps^2."""
    for act in ("silu", "gelu", "none"):
        g = gen(6)
        m, d, f = 33, 72, 90
        x, wg, wu = rows(g, m, d, 1.0, BF, "cuda"), rows(g, f, d, 0.1, BF, "cuda"), rows(g, f, d, 0.1, BF, "cuda")
        dh = rows(g, m, f, 1.0, BF, "cuda", pad=1)
        grads = kd.gated_ffn_backward(x, wg, wu, dh, act=act)
        base = [t.double() for t in (x, wg, wu)]

        def loss(p):
            return (dh.double() * act64(act, p[0] @ p[1].t()) * (p[0] @ p[2].t())).sum()

        for i in range(3):
            v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
            eps = 1e-5
            up, down = [list(base) for _ in range(2)]
            up[i], down[i] = base[i] + eps * v, base[i] - eps * v
            want = float((loss(up) - loss(down)) / (2 * eps))
            got = float((grads[i].double() * v).sum())
            assert abs(got - want) <= 2 * half_step(BF) * float(grads[i].double().norm() * v.norm()) + 1e-6 * abs(want), (act, i)
