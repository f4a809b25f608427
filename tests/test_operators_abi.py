"""The prompt operators' refusals and workspace sizes, without a GPU: arguments are checked on the
host before a device is touched."""

import pytest
import torch

import synth
from persistent_monokernel_sm_b200 import build

build.build()
import persistent_monokernel_sm_b200 as kd  # noqa: E402

P = 1 << 20  # an aligned address that nothing reads


def linear(**kw):
    a = dict(dtype=0, out_dtype=0, act=0, w_transposed=0, m=4, n=16, k=32, x=P, ld_x=32, w=P, ld_w=32, bias=None,
             residual=None, ld_residual=0, out=P, ld_out=16)
    a.update(kw)
    return kd.load_library().kd_linear(bytes(kd.kd_linear_args(**a)), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(out_dtype=1), dict(out_dtype=3), dict(act=4), dict(act=-1), dict(w_transposed=2),
    dict(m=-1), dict(n=-1), dict(k=0), dict(k=-5), dict(m=1 << 31), dict(n=1 << 40), dict(x=None), dict(w=None), dict(out=None),
    dict(x=P + 2), dict(w=P + 8), dict(ld_x=31), dict(ld_x=36), dict(ld_w=24), dict(ld_w=36), dict(ld_x=1 << 39),
    dict(out=P + 1), dict(ld_out=15), dict(bias=P + 1), dict(residual=P + 1, ld_residual=16), dict(residual=P, ld_residual=8),
    dict(out_dtype=2, out=P + 2), dict(w_transposed=1, ld_w=8), dict(w_transposed=1, ld_w=20)])
def test_linear_refuses(bad):
    assert linear(**bad) == -1
    assert len(kd.kd_op_error()) > 5


def test_nothing_to_do_is_no_error():
    assert linear(m=0) == 0
    assert linear(n=0, ld_out=0) == 0
    assert gated(m=0) == 0 and gated(f=0) == 0
    assert attention(n=0) == 0
    assert kd.load_library().kd_linear(None, None) == -1


def gated(h=P, ld_h=48, **kw):
    a = dict(dtype=0, act=2, m=4, d=32, f=48, x=P, ld_x=32, wg=P, ld_wg=32, wu=P, ld_wu=64)
    a.update(kw)
    return kd.load_library().kd_gated_ffn(bytes(kd.kd_gated_args(**a)), h, ld_h, None)


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(act=9), dict(m=-1), dict(d=0), dict(f=-2), dict(x=None), dict(wg=None),
                                 dict(wu=None), dict(x=P + 4), dict(wu=P + 2), dict(ld_x=30), dict(ld_wg=20), dict(ld_wu=33),
                                 dict(h=None), dict(h=P + 1), dict(ld_h=47)])
def test_gated_refuses(bad):
    assert gated(**bad) == -1


def backward(args=None, dh=P, ld_dh=48, dx=P, ld_dx=32, dwg=P, ld_dwg=32, dwu=P, ld_dwu=32, ws=P, size=None, **kw):
    a = dict(dtype=0, act=2, m=4, d=32, f=48, x=P, ld_x=32, wg=P, ld_wg=32, wu=P, ld_wu=64)
    a.update(kw)
    size = kd.kd_gated_ffn_backward_workspace(a["m"], a["f"]) if size is None else size
    return kd.load_library().kd_gated_ffn_backward(bytes(kd.kd_gated_args(**a)), dh, ld_dh, dx, ld_dx, dwg, ld_dwg, dwu, ld_dwu,
                                                   ws, size, None)


@pytest.mark.parametrize("bad,code", [(dict(m=0), -1), (dict(f=0), -1), (dict(dh=None), -1), (dict(ld_dh=40), -1),
                                      (dict(ld_dx=31), -1), (dict(ld_dwg=8), -1), (dict(ld_dwu=8), -1), (dict(dx=P + 1), -1),
                                      (dict(ws=None), -2), (dict(size=100), -2), (dict(x=P + 2), -1)])
def test_backward_refuses(bad, code):
    assert backward(**bad) == code


def attention(**kw):
    a = dict(dtype=0, n_heads=4, n_kv_heads=2, head_dim=64, n=3, kv_len=5, q=P, q_token=256, q_head=64, k=P, k_pos=64, k_head=6400,
             v=P, v_pos=64, v_head=6400, out=P, out_token=256, out_head=64, scale=0.125, workspace=None, workspace_bytes=0)
    a.update(kw)
    return kd.load_library().kd_prompt_attention(bytes(kd.kd_attention_args(**a)), None)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), -1), (dict(head_dim=96), -1), (dict(n_heads=3), -1), (dict(n_heads=0), -1), (dict(n_kv_heads=0), -1),
    (dict(n_heads=258, n_kv_heads=2), -1), (dict(n=-1), -1), (dict(kv_len=-1), -1), (dict(kv_len=1 << 30), -1), (dict(q=None), -1),
    (dict(k=P + 8), -1), (dict(v=P + 2), -1), (dict(out=P + 4), -1), (dict(q_token=60), -1), (dict(k_pos=68), -1), (dict(v_head=12), -1),
    (dict(out_head=1 << 39), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(kv_len=4000), -2), (dict(kv_len=4000, workspace=P, workspace_bytes=1000), -2)])
def test_attention_refuses(bad, code):
    assert attention(**bad) == code


def test_workspaces():
    a = kd.kd_attention_args(dtype=0, n_heads=16, n_kv_heads=8, head_dim=128, n=1, kv_len=0, scale=1.0)
    assert kd.kd_prompt_attention_workspace(a) == 0
    most = 0
    for kv in (100, 300, 1000, 5000, 32768, 1 << 20):
        for n in (1, 7, 100, 1000, 20000):
            for hq, hkv in ((1, 1), (8, 1), (16, 8), (12, 4)):
                a.n, a.kv_len, a.n_heads, a.n_kv_heads = n, kv, hq, hkv
                size = kd.kd_prompt_attention_workspace(a)
                if n * hq > 128 * 148:
                    assert size == 0
                most = max(most, size)
    assert 0 < most <= 148 * 128 * 132 * 4 + 256
    a.head_dim = 96
    assert kd.kd_prompt_attention_workspace(a) == 0
    assert kd.kd_gated_ffn_backward_workspace(10, 100) >= 2 * 10 * 100 * 2
    assert kd.kd_gated_ffn_backward_workspace(-1, 100) == 0
    cfg = kd.config_from(synth.get("tiny").dims(), 64)
    sizes = [kd.kd_prefill_workspace(cfg, n) for n in (1, 16, 1000)]
    assert 0 < sizes[0] < sizes[1] < sizes[2]
    assert kd.kd_prefill_workspace(cfg, 0) == 0
    cfg.head_dim = 96
    assert kd.kd_prefill_workspace(cfg, 16) == 0
    assert kd.load_library().kd_prefill(None, None, 1, 0, None, 0) == -1


def test_tensors_are_checked():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: kd.linear(x, w), lambda: kd.linear(None, w), lambda: kd.linear([1], w), lambda: kd.gated_ffn(x, w, w),
                 lambda: kd.gated_ffn_backward(x, w, w, x), lambda: kd.prompt_attention(x[None], x[None], x[None], 0)):
        with pytest.raises(kd.KdError) as e:
            call()
        assert e.value.code == -1
        assert len(str(e.value)) > 20
    with pytest.raises(TypeError):
        kd.linear(x)
