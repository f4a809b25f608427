"""A device-side wait of kd_prefill that exceeds the handle's limit is the handle's error: kd_sync reports
it, kd_decode is refused until a reset, and with the limit back the request runs as before."""

import numpy as np
import pytest
import torch

import persistent_monokernel_sm_b200 as kd
import synth

pytestmark = pytest.mark.gpu


def make(name, n, **kw):
    w = synth.get(name).replace(kv_len=0, **kw)
    dec = kd.Decoder(w.dims(), n + 8)
    dec.load_weights(synth.make_weights(w, seed=0, device="cuda"))
    return dec, np.random.RandomState(0).randint(0, w.vocab, n)


def caches(dec, dims, n, cap):
    out = []
    for l in range(dims["n_layers"]):
        for s in (0, 1):
            off = kd.kd_kv_ptr(dec.h, l, s) - dec.arena.data_ptr()
            size = dims["n_kv_heads"] * cap * dims["head_dim"] * 2
            out.append(dec.arena[off:off + size].view(torch.bfloat16).view(dims["n_kv_heads"], cap, dims["head_dim"])[:, :n].clone())
    return out


# the second runs with pairs of CTAs and whole attention tiles
@pytest.mark.parametrize("name,n,kw", [("tiny", 150, {}), ("2b-4k", 2500, dict(n_layers=2, vocab=1000))])
@pytest.mark.parametrize("decode", [False, True])
def test_a_wait_that_runs_out(name, n, kw, decode):
    dec, prompt = make(name, n, **kw)
    dec.prefill(prompt)
    want = caches(dec, dec.dims, n - 1, n + 8)
    _, lg = dec.decode(1, logits=True)
    dec.sync()
    for _ in range(2):
        kd.kd_set_timeout(dec.h, 1)
        dec.prefill(prompt)
        kd.kd_set_timeout(dec.h, 1_000_000_000)
        if decode:
            dec.decode(4)  # enqueued before anybody knows: it stops too
        with pytest.raises(kd.KdError) as e:
            dec.sync()
        assert e.value.code == -6 and "kind 7" in str(e.value)
        with pytest.raises(kd.KdError) as e:
            dec.decode(1)
        assert e.value.code == -7
        kd.kd_op_sync(dec.stream.cuda_stream)  # no error of the operators called by themselves
        dec.prefill(prompt)
        assert all(torch.equal(a, b) for a, b in zip(want, caches(dec, dec.dims, n - 1, n + 8)))
        _, again = dec.decode(1, logits=True)
        dec.sync()
        # the decode launch's sums over CTAs are taken in the order of their arrival
        assert float((again - lg).norm()) <= 1e-4 * float(lg.norm())
    dec.close()


def test_the_operators_limit_is_not_the_handles():
    dec, prompt = make("tiny", 60)
    kd.kd_op_set_timeout(1)
    try:
        dec.prefill(prompt)
        dec.decode(2)
        dec.sync()
    finally:
        kd.kd_op_set_timeout(2_000_000_000)
    kd.kd_op_sync(dec.stream.cuda_stream)
    dec.close()
