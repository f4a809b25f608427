"""The prompt operators' cases: what is measured, their plain forms and their 64-bit values.

Operators (a prompt's tokens, or one token, through one layer of the decoder):

* ``linear``    out = residual + act(x W^T + bias): the Q/K/V, output and down projections, the LM head
* ``gated``     h = act(x Wg^T) * (x Wu^T): the feed-forward block's two projections, activation and product
* ``gated_bwd`` its gradients dx, dWg, dWu for a given dh, recomputing both projections
* ``attention`` causal attention of n new tokens over a key-value cache of kv_len earlier positions
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_lib = None


def _kd():
    global _lib
    if _lib is None:
        import persistent_monokernel_sm_b200 as kd
        _lib = kd
    return _lib


def listed():
    return [
        # one token's output projection of the 0.5B model, added to the fp32 residual: latency
        dict(name="linear_one_token", op="linear", m=1, n=1536, k=1536, w_t=False, bias=False, act="none",
             res="f32", out="f32", dtype="bf16"),
        # a 128-token prompt's down projection of the 0.5B model, from the weight laid out [in][out]
        dict(name="linear_prompt_down", op="linear", m=128, n=1536, k=4096, w_t=True, bias=False, act="none",
             res="f32", out="f32", dtype="bf16"),
        # one token's LM head of the 8B model: a gigabyte of weights read once
        dict(name="linear_lm_head", op="linear", m=1, n=128256, k=4096, w_t=False, bias=False, act="none",
             res="none", out="f32", dtype="bf16"),
        # a long prompt of odd length through a projection with bias and activation
        dict(name="linear_long_bias_gelu", op="linear", m=4095, n=8192, k=2048, w_t=False, bias=True, act="gelu",
             res="none", out="bf16", dtype="bf16"),
        # one token through the 0.5B model's feed-forward block: latency
        dict(name="gated_one_token", op="gated", m=1, d=1536, f=4096, act="silu", dtype="bf16"),
        # a 128-token prompt through the 2B model's
        dict(name="gated_prompt", op="gated", m=128, d=2048, f=8192, act="silu", dtype="bf16"),
        # a 4,096-token prompt through the 8B model's
        dict(name="gated_long", op="gated", m=4096, d=4096, f=14336, act="silu", dtype="bf16"),
        # a small ragged training batch, a hidden width of odd size, fp16
        dict(name="gated_bwd_ragged", op="gated_bwd", m=257, d=256, f=1001, act="gelu", dtype="f16"),
        # a training batch of the 2B model's block
        dict(name="gated_bwd_long", op="gated_bwd", m=4096, d=2048, f=8192, act="silu", dtype="bf16"),
        # one token at the end of the 2B model's 32k cache
        dict(name="attention_one_token_32k", op="attention", n=1, kv_len=32768, hq=16, hkv=8, hd=128, dtype="bf16"),
        # a 4,096-token prompt of the 8B model from an empty cache
        dict(name="attention_long_prompt", op="attention", n=4096, kv_len=0, hq=32, hkv=8, hd=128, dtype="bf16"),
        # a piece of odd length behind a prefix, heads of 64
        dict(name="attention_ragged_chunk", op="attention", n=77, kv_len=1001, hq=4, hkv=2, hd=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated_bwd", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "linear":
        out = rng.choice(["same", "f32"])
        out = dtype if out == "same" else out
        n, k = _log(rng, 64, 16384), _log(rng, 64, 14336)
        m = _log(rng, 1, max(1, min(4096, int(6.8e10 / (n * k)))))
        return dict(op=op, m=m, n=n, k=k, w_t=rng.random() < 0.4, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "none", "relu", "silu", "gelu"]), res=rng.choice(["none", out]),
                    out=out, dtype=dtype)
    if op in ("gated", "gated_bwd"):
        d, f = 8 * _log(rng, 8, 512), _log(rng, 64, 14336)
        most = (2.2e11 if op == "gated" else 6e10) / (d * f)
        return dict(op=op, m=_log(rng, 1, max(1, min(4096, int(most)))), d=d, f=f,
                    act=rng.choice(["silu", "gelu", "relu"]), dtype=dtype)
    hd, hkv, r = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    n = _log(rng, 1, 4096)
    most = min(32768, int(4e8 / (n * hkv * r)))
    kv_len = rng.choice([0, max(0, _log(rng, 1, max(1, most)) - n)])
    return dict(op=op, n=n if kv_len else min(n, most), kv_len=kv_len, hq=hkv * r, hkv=hkv, hd=hd, dtype=dtype)


def _rows(g, rows, cols, scale, dt, pad=8):
    """[rows][cols] of N(0, scale) whose rows start on a multiple of `pad` elements."""
    ld = -(-cols // pad) * pad
    t = torch.randn(rows, ld, generator=g, device="cuda", dtype=torch.float32 if rows * ld < 1 << 27 else dt)
    return t.mul_(scale).to(dt)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    dt = _DT[case["dtype"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _rows(g, m, k, 1.0, dt)                                          # a normalised activation
        s["w"] = _rows(g, k, n, 0.02, dt) if case["w_t"] else _rows(g, n, k, 0.02, dt)
        s["b"] = torch.randn(n, generator=g, device="cuda").mul_(0.1).to(dt) if case["bias"] else None
        s["r"] = _rows(g, m, n, 1.0, _DT[case["res"]], 1) if case["res"] != "none" else None
    elif case["op"] in ("gated", "gated_bwd"):
        m, d, f = case["m"], case["d"], case["f"]
        s["x"] = _rows(g, m, d, 1.0, dt)
        s["wg"] = _rows(g, f, d, 0.02, dt)
        s["wu"] = _rows(g, f, d, 0.02, dt)
        if case["op"] == "gated_bwd":
            s["dh"] = _rows(g, m, f, 0.1, dt, 1)
    else:
        n, T, hd = case["n"], case["n"] + case["kv_len"], case["hd"]
        cap = -(-T // 64) * 64 + 64                                               # the cache holds more than is filled
        s["q"] = torch.randn(n, case["hq"], hd, generator=g, device="cuda").to(dt)
        s["k"] = torch.randn(case["hkv"], cap, hd, generator=g, device="cuda").to(dt)
        s["v"] = torch.randn(case["hkv"], cap, hd, generator=g, device="cuda").to(dt)
    return s


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z * (z > 0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327


def run(s):
    op = s["op"]
    if own:
        kd = _kd()
        if op == "linear":
            return kd.linear(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["r"], out_dtype=_DT[s["out"]],
                             w_t=s["w_t"])
        if op == "gated":
            return kd.gated_ffn(s["x"], s["wg"], s["wu"], act=s["act"])
        if op == "gated_bwd":
            return kd.gated_ffn_backward(s["x"], s["wg"], s["wu"], s["dh"], act=s["act"])
        return kd.prompt_attention(s["q"], s["k"], s["v"], s["kv_len"])
    dt = _DT[s["dtype"]]
    if op == "linear":
        w = s["w"].float()
        y = s["x"].float() @ (w if s["w_t"] else w.t())
        if s["b"] is not None:
            y = y + s["b"].float()
        y = _act(s["act"], y)
        if s["r"] is not None:
            y = y + s["r"].float()
        return y.to(_DT[s["out"]])
    if op == "gated":
        x = s["x"].float()
        return (_act(s["act"], x @ s["wg"].float().t()) * (x @ s["wu"].float().t())).to(dt)
    if op == "gated_bwd":
        x, wg, wu, dh = s["x"].float(), s["wg"].float(), s["wu"].float(), s["dh"].float()
        g, u = x @ wg.t(), x @ wu.t()
        dg, du = dh * u * _slope(s["act"], g), dh * _act(s["act"], g)
        return (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    n, T, hkv, hd = s["n"], s["n"] + s["kv_len"], s["hkv"], s["hd"]
    r = s["hq"] // hkv
    q = s["q"].float().view(n, hkv, r, hd).permute(1, 2, 0, 3).reshape(hkv, r * n, hd)
    z = (q @ s["k"][:, :T].float().transpose(1, 2)).mul_(1 / math.sqrt(hd)).view(hkv, r, n, T)
    late = torch.arange(T, device=z.device)[None, :] > s["kv_len"] + torch.arange(n, device=z.device)[:, None]
    z.masked_fill_(late, -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    z = z / z.sum(-1, keepdim=True)
    y = z.view(hkv, r * n, T) @ s["v"][:, :T].float()
    return y.view(hkv, r, n, hd).permute(2, 0, 1, 3).reshape(n, hkv * r, hd).to(dt)


def work(case):
    e = 2
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        size = {"none": 0, "bf16": 2, "f16": 2, "f32": 4}
        return {"bytes": e * (m * k + n * k + n * case["bias"]) + m * n * (size[case["res"]] + size[case["out"]]),
                "flops": 2 * m * n * k}
    if case["op"] in ("gated", "gated_bwd"):
        m, d, f = case["m"], case["d"], case["f"]
        once = e * (m * d + 2 * f * d + m * f)
        if case["op"] == "gated":
            return {"bytes": once, "flops": 4 * m * d * f}
        return {"bytes": once + e * (m * d + 2 * f * d), "flops": 12 * m * d * f}
    n, p, hq, hkv, hd = (case[c] for c in ("n", "kv_len", "hq", "hkv", "hd"))
    return {"bytes": e * (2 * n * hq * hd + 2 * hkv * (p + n) * hd),
            "flops": 4 * hd * hq * (n * p + n * (n + 1) // 2)}


def exact(case, seed):
    s = prepare(case, seed)
    up = lambda t: t.to(torch.float64)  # noqa: E731
    phi = lambda z: torch.special.ndtr(z)  # noqa: E731
    f = {"none": lambda z: z, "relu": lambda z: torch.clamp(z, min=0), "silu": lambda z: z * torch.sigmoid(z),
         "gelu": lambda z: z * phi(z)}
    op = case["op"]
    if op == "linear":
        x, w = up(s["x"]), s["w"].t() if case["w_t"] else s["w"]
        parts = [x @ up(w[i:i + 16384]).t() for i in range(0, case["n"], 16384)]
        y = torch.cat(parts, 1)
        y = f[case["act"]](y if s["b"] is None else y + up(s["b"]))
        return y if s["r"] is None else y + up(s["r"])
    if op in ("gated", "gated_bwd"):
        x, wg, wu = up(s["x"]), up(s["wg"]), up(s["wu"])
        g, u = torch.einsum("md,fd->mf", x, wg), torch.einsum("md,fd->mf", x, wu)
        if op == "gated":
            return f[case["act"]](g) * u
        dh = up(s["dh"])
        slope = {"relu": lambda z: (z > 0).double(),
                 "silu": lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z),
                 "gelu": lambda z: phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[case["act"]]
        dg, du = dh * u * slope(g), dh * f[case["act"]](g)
        return (torch.einsum("mf,fd->md", dg, wg) + torch.einsum("mf,fd->md", du, wu),
                torch.einsum("mf,md->fd", dg, x), torch.einsum("mf,md->fd", du, x))
    n, p, r = case["n"], case["kv_len"], case["hq"] // case["hkv"]
    y = torch.empty(n, case["hq"], case["hd"], dtype=torch.float64, device="cuda")
    at = torch.arange(p, p + n, device="cuda")
    for h in range(case["hq"]):
        k, v = up(s["k"][h // r, :p + n]), up(s["v"][h // r, :p + n])
        z = torch.einsum("nd,td->nt", up(s["q"][:, h]), k) / np.sqrt(float(case["hd"]))
        z = torch.where(torch.arange(p + n, device="cuda")[None] <= at[:, None], z, -math.inf)
        y[:, h] = torch.softmax(z, -1) @ v
    return y
