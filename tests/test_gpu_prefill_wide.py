"""kd_prefill at the widths of the 2B and 8B models (two layers, a small vocabulary) and at lengths where
pairs of CTAs, 256-column tiles, whole attention tiles and several pieces run, against 64 bits; and greedy
tokens after a prefill, with prompts chosen so that the comparison always takes place."""

import numpy as np
import pytest
import torch

import persistent_monokernel_sm_b200 as kd
import synth
from tests.test_gpu_prefill import forward, run, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,n,max_piece", [("2b-4k", 2049, 4096), ("2b-4k", 1300, 500), ("8b-4k", 1025, 4096), ("0.5b", 1200, 4096)])
def test_wide_layers_and_long_prompts(name, n, max_piece):
    w = synth.get(name).replace(n_layers=2, vocab=1000, kv_len=0)
    run(w, synth.make_weights(w, seed=0, device="cuda"), np.random.RandomState(n).randint(0, w.vocab, n), None, max_piece)


def test_greedy_token_after_a_prefill():
    """The bars of the other tests on the logits, |prefill - plain| <= 2 |rounded - plain| and |decode - plain| <=
    1e-3 |plain|, bound how far the two ways' logits are apart; prompts whose top two differ by more than twice
    that have to give the same token."""
    w = synth.get("tiny").replace(vocab=32)
    W = weights(w)
    dims = w.dims()
    dec = kd.Decoder(dims, 200)
    dec.load_weights(W)
    compared = 0
    for seed in range(40):
        prompt = np.random.RandomState(100 + seed).randint(0, w.vocab, 120)
        plain, rounded = forward(dims, W, prompt, False)[2][0], forward(dims, W, prompt, True)[2][0]
        may = 2 * float((rounded - plain).norm()) + 1e-3 * float(plain.norm())
        dec.reset(prompt, 0)
        slow, lg_slow = dec.decode(1, logits=True)
        dec.sync()
        dec.prefill(prompt)
        fast, lg_fast = dec.decode(1, logits=True)
        dec.sync()
        assert float((lg_slow[-1] - lg_fast[-1]).norm()) <= may
        top = torch.topk(plain, 2).values
        if float(top[0] - top[1]) > 2 * may:
            compared += 1
            assert int(slow[0]) == int(fast[0]) == int(plain.argmax())
        if compared == 5:
            break
    assert compared == 5, compared
    dec.close()
