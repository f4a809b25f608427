"""Decoder.prefill on a stream of its own, with tokens that lie on the GPU and belong to another stream: it
waits for what makes them, and their memory is not given away before it has read them."""

import numpy as np
import pytest
import torch

import persistent_monokernel_sm_b200 as kd
import synth

pytestmark = pytest.mark.gpu
N = 90


@pytest.fixture
def dec():
    w = synth.get("tiny")
    d = kd.Decoder(w.dims(), 4 * N, stream=torch.cuda.Stream())
    d.load_weights(synth.make_weights(w, seed=0, device="cpu"))
    yield d
    d.close()


def prompt(seed):
    return torch.as_tensor(np.random.RandomState(seed).randint(1, 4096, N), dtype=torch.int32)


def cache(dec, n):
    dec.stream.synchronize()
    out = []
    for l in range(dec.dims["n_layers"]):
        for s in (0, 1):
            off = kd.kd_kv_ptr(dec.h, l, s) - dec.arena.data_ptr()
            t = dec.arena[off:off + 2 * 4 * N * 64 * 2].view(torch.bfloat16).view(2, 4 * N, 64)
            out.append(t[:, :n].clone())
    return out


def test_tokens_that_another_stream_is_still_making(dec):
    dec.prefill(prompt(0))
    want = cache(dec, N - 1)
    made, t = prompt(0).cuda(), torch.zeros(N, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    t.copy_(made)
    dec.prefill(t)
    dec.sync()
    assert all(torch.equal(a, b) for a, b in zip(want, cache(dec, N - 1)))


def test_tokens_whose_memory_is_used_again(dec):
    dec.prefill(prompt(1))
    want = cache(dec, N - 1)
    before, t, later = prompt(3).cuda(), prompt(1).cuda(), prompt(2).cuda()  # what the middle one leaves is a hole
    at = t.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(dec.stream):
        torch.cuda._sleep(600_000_000)
    dec.prefill(t)
    del t
    dec.prefill(later, kv_len=N)  # the handle lets the first tokens go
    others = [torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(64)]  # takes such holes first
    assert not dec.stream.query()  # the tokens have not been read yet
    assert all(o.data_ptr() != at for o in others)
    dec.sync()
    assert all(torch.equal(a, b) for a, b in zip(want, cache(dec, N - 1)))
    assert before.numel() == N
