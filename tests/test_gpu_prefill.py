"""kd_prefill on the GPU: the operators run together through a model's layers.

Two float64 references, both the definition of the decoder: `plain` with no rounding but the
cache's, and `rounded` with the bf16 roundings that kd_prefill documents (normalised activations,
q, attention outputs, hidden units) at the same places. kd_prefill computes the latter in fp32
sums, so it has to be as near to `plain` as `rounded` is, up to a factor of 2 (a rounding may fall
to the other neighbour where two sums differ in their last bits), in every layer's cache rows
and in the logits that the decode launch forms from them."""

import math

import numpy as np
import pytest
import torch

import persistent_monokernel_sm_b200 as kd
import synth

pytestmark = pytest.mark.gpu


def forward(dims, W, tokens, rounded, prefix=None):
    """(K, V [L][Hkv][n][hd], logits of the last token) in float64 on the GPU. As in the call, the last
    token goes through without the extra roundings."""
    L, Hq, Hkv, hd = dims["n_layers"], dims["n_heads"], dims["n_kv_heads"], dims["head_dim"]
    n, p = len(tokens), 0 if prefix is None else prefix[0].shape[2]
    up = lambda t: t.cuda().double()  # noqa: E731
    bf = lambda t: t.float().to(torch.bfloat16).double()  # noqa: E731

    def rnd(t):
        return torch.cat([bf(t[:-1]), t[-1:]]) if rounded else t

    def rms(x, g):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + float(dims["rms_eps"])) * up(g)

    freq = float(dims["rope_theta"]) ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device="cuda") / hd)
    ang = torch.arange(p, p + n, dtype=torch.float64, device="cuda")[:, None] * freq
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def rope(x):
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = up(W["embed"])[torch.as_tensor(np.asarray(tokens, np.int64), device="cuda")]
    mask = torch.arange(p + n, device="cuda")[None] <= p + torch.arange(n, device="cuda")[:, None]
    Ks, Vs = [], []
    for l in range(L):
        xn = rnd(rms(x, W["attn_norm"][l]))
        q = rnd(rope((xn @ up(W["wq"][l]).T).view(n, Hq, hd)))
        k = bf(rope((xn @ up(W["wk"][l]).T).view(n, Hkv, hd))).transpose(0, 1)
        v = bf((xn @ up(W["wv"][l]).T).view(n, Hkv, hd)).transpose(0, 1)
        Ks.append(k)
        Vs.append(v)
        if prefix is not None:
            k, v = torch.cat([up(prefix[0][l]), k], 1), torch.cat([up(prefix[1][l]), v], 1)
        o = torch.empty(n, Hq, hd, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            z = (q[:, h] @ k[h * Hkv // Hq].T / math.sqrt(hd)).masked_fill(~mask, float("-inf"))
            o[:, h] = torch.softmax(z, 1) @ v[h * Hkv // Hq]
        x = x + rnd(o.view(n, Hq * hd)) @ up(W["wo"][l]).T
        xn = rnd(rms(x, W["ffn_norm"][l]))
        g = xn @ up(W["wg"][l]).T
        x = x + rnd(g * torch.sigmoid(g) * (xn @ up(W["wu"][l]).T)) @ up(W["wd"][l]).T
    return torch.stack(Ks), torch.stack(Vs), rms(x[-1:], W["final_norm"]) @ up(W["lm_head"]).T


def cache_rows(dec, dims, layer, which, lo, hi, cap):
    """[Hkv][hi - lo][hd] of the handle's cache, as a tensor view of the arena."""
    off = kd.kd_kv_ptr(dec.h, layer, which) - dec.arena.data_ptr()
    size = dims["n_kv_heads"] * cap * dims["head_dim"] * 2
    t = dec.arena[off:off + size].view(torch.bfloat16).view(dims["n_kv_heads"], cap, dims["head_dim"])
    return t[:, lo:hi]


def run(w, W, tokens, prefix=None, max_piece=4096, spare=3):
    dims, n, p = w.dims(), len(tokens), 0 if prefix is None else prefix[0].shape[2]
    cap = p + n + spare
    dec = kd.Decoder(dims, cap)
    dec.load_weights(W)
    for l in range(dims["n_layers"]):  # what the cache holds before it is written
        for s in (0, 1):
            cache_rows(dec, dims, l, s, 0, cap, cap).fill_(float("nan"))
    if prefix is not None:
        dec.set_kv(*prefix)
    launches = dec.info().launches
    dec.prefill(tokens, p, max_piece)
    assert dec.position() == p + n - 1
    pieces, least = -(-(n - 1) // max_piece), 8 * dims["n_layers"] - 5  # and a join where attention is split
    assert least * pieces <= dec.info().launches - launches <= (least + dims["n_layers"] - 1) * pieces
    before = [cache_rows(dec, dims, l, s, p, p + n - 1, cap).clone() for l in range(dims["n_layers"]) for s in (0, 1)]
    _, lg = dec.decode(1, logits=True)
    dec.sync()
    kd.kd_op_sync(dec.stream.cuda_stream)
    plain = forward(dims, W, tokens, False, prefix)
    rounded = forward(dims, W, tokens, True, prefix)
    for l in range(dims["n_layers"]):
        for s in (0, 1):
            got = before[2 * l + s].double()
            a, b = plain[s][l][:, :-1], rounded[s][l][:, :-1]
            assert bool(torch.isfinite(got).all())
            if n > 1:
                far, may = (got - a).norm() / a.norm(), (b - a).norm() / a.norm()
                # layer 0's rows differ from `plain` by the rounding of xn alone
                assert far <= 2 * may, ("KV"[s], l, float(far), float(may))
    far, may = (lg[0].double() - plain[2][0]).norm(), (rounded[2][0] - plain[2][0]).norm()
    # with nothing prefilled the logits are the decode launch's own: its bar of 1e-3
    assert far <= max(2 * float(may), 1e-3 * float(plain[2].norm())), (float(far), float(may))
    dec.close()
    return lg


def weights(w, seed=0):
    return synth.make_weights(w, seed=seed, device="cpu" if w.d_model <= 1536 else None)


@pytest.mark.parametrize("n", [1, 2, 3, 17, 130, 300])
def test_tiny_prompts(n):
    w = synth.get("tiny")
    run(w, weights(w), np.random.RandomState(n).randint(0, w.vocab, n))


@pytest.mark.parametrize("max_piece", [1, 7, 64])
def test_pieces_and_prefix(max_piece):
    w = synth.get("tiny").replace(kv_len=70)
    K, V = synth.make_kv(w, seed=2, device="cpu")
    run(w, weights(w), np.random.RandomState(5).randint(0, w.vocab, 41 if max_piece > 1 else 6), (K, V), max_piece)


def test_odd_hidden_width_and_groups_of_three():
    w = synth.get("tiny").replace(n_heads=6, n_kv_heads=2, ffn_dim=1003, head_dim=128)
    run(w, weights(w), np.random.RandomState(9).randint(0, w.vocab, 150))


def test_half_billion_prompt():
    w = synth.get("0.5b")
    W = weights(w)
    run(w, W, synth.make_prompt(w).numpy())


def test_decode_continues_and_a_second_request_follows():
    """Greedy tokens after kd_prefill equal those after the token-by-token prompt wherever the
    margin of the top two logits is above what the roundings can move."""
    w = synth.get("tiny")
    W = weights(w)
    dec = kd.Decoder(w.dims(), 400)
    dec.load_weights(W)
    prompt = np.random.RandomState(3).randint(0, w.vocab, 120)
    for _ in range(2):
        dec.reset(prompt, 0)
        slow, lg_slow = dec.decode(1, logits=True)
        dec.sync()
        dec.prefill(prompt)
        fast, lg_fast = dec.decode(1, logits=True)
        dec.sync()
        a, b = lg_slow[-1], lg_fast[-1]
        top = torch.topk(a, 2).values
        if float(top[0] - top[1]) > 2 * float((a - b).abs().max()):
            assert int(slow[0]) == int(fast[0])
    more, _ = dec.decode(20)
    dec.sync()
    assert dec.position() == 120 + 20
    assert int(more.min()) >= 0 and int(more.max()) < w.vocab


def test_bad_token_is_reported_and_the_handle_recovers():
    w = synth.get("tiny")
    dec = kd.Decoder(w.dims(), 64)
    dec.load_weights(weights(w))
    for bad in (w.vocab, -1):
        dec.prefill([1, 2, bad, 3, 4])
        with pytest.raises(kd.KdError) as e:
            dec.sync()
        assert e.value.code == -8
    dec.prefill([1, 2, 3, 4])
    dec.decode(2)
    dec.sync()


def test_refusals():
    w = synth.get("tiny")
    dec = kd.Decoder(w.dims(), 64)
    with pytest.raises(kd.KdError) as e:
        dec.prefill([1, 2, 3])
    assert e.value.code == -7  # no weights
    dec.load_weights(weights(w))
    t = torch.arange(65, dtype=torch.int32, device="cuda")
    ws = torch.empty(2048, dtype=torch.uint8, device="cuda")
    for args, code in (((t.data_ptr(), 65, 0), -3), ((t.data_ptr(), 5, 60), -3), ((t.data_ptr(), 0, 0), -1), ((None, 3, 0), -1),
                       ((t.data_ptr(), 3, -1), -1), ((t.data_ptr(), 3, 0), -2)):
        with pytest.raises(kd.KdError) as e:
            kd.kd_prefill(dec.h, *args, ws.data_ptr(), 2048)
        assert e.value.code == code, args
