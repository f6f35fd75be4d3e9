"""Beam search over a hybrid model (modal Hyena and linear attention), end to end.

Each sequence found is scored again without a search: prompt and sequence as one
prompt through the prefill path, the log probabilities of its tokens summed in
float64.  Nothing there reorders a state, so a beam that went on with another
beam's state would not agree.

Tolerance.  The two paths round the same values to bfloat16 at the same places but
sum in another order, so an activation may land on the neighbouring bfloat16 value
(2^-8 of it); with L layers of two products, sign-random, a logit of size up to 12
moves by some 12 * 2^-8 * sqrt(2 L) / 3 = 0.05 for L = 4, its log probability by
twice that at most: 0.1 a token.  A state of another beam moves it by units.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu


def _model(torch, **kw):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from beam_generate import random_model
    return random_model(torch, **kw)


@pytest.mark.parametrize("G,K,L,steps,end", [(1, 4, 5, 12, None), (3, 5, 90, 9, None), (2, 4, 40, 10, 7)])
def test_sequences_score_as_prompts(G, K, L, steps, end):
    torch = require_gpu()
    V = 600
    model = _model(torch, layers=4, width=128, vocab=V, heads=4, modes=8, seed=G)
    prompts = torch.randint(0, V, (G, L), generator=torch.Generator().manual_seed(L)).cuda()
    if end is not None:  # an end that is found now and then
        model.head[end] *= 0.0
        model.head[end] += model.head[11]
    log(f"hybrid beams {G}x{K}, {L}+{steps}")
    tokens, scores = model.generate(prompts, K, steps, end_token=end)
    torch.cuda.synchronize()
    assert tokens.shape == (G, K, steps) and scores.shape == (G, K)
    assert bool((scores[:, :-1] >= scores[:, 1:]).all())
    seqs = {tuple(t) for t in tokens.reshape(G * K, steps).tolist()}
    assert len(seqs) > G * K // 2
    whole = torch.cat([prompts.repeat_interleave(K, 0), tokens.reshape(G * K, steps).long()], 1)
    logits, _ = model.prefill(whole)
    logp = torch.log_softmax(logits.view(G * K, L + steps, V).double(), -1)[:, L - 1:-1]
    each = logp.gather(2, tokens.reshape(G * K, steps, 1).long())[..., 0].cpu().numpy()
    got = tokens.reshape(G * K, steps).cpu().numpy()
    want = np.zeros(G * K)
    for r in range(G * K):
        for t in range(steps):
            want[r] += each[r, t]
            if end is not None and got[r, t] == end:
                assert (got[r, t:] == end).all()
                break
    off = abs(scores.reshape(-1).cpu().numpy() - want)
    assert off.max() <= 0.1 * steps, off


def test_one_beam_is_greedy():
    """One beam takes the likeliest token each time, as a loop over prefills does (ties aside)."""
    torch = require_gpu()
    model = _model(torch, layers=2, width=64, vocab=300, heads=2, modes=8, seed=5)
    seq = torch.randint(0, 300, (2, 20), generator=torch.Generator().manual_seed(3)).cuda()
    log("hybrid greedy")
    tokens, _ = model.generate(seq, 1, 5)
    for t in range(5):
        logits, _ = model.prefill(seq)
        last = logits.view(2, seq.shape[1], -1)[:, -1].float()
        picked = last.gather(1, tokens[:, 0, t:t + 1].long())[:, 0]
        assert bool((picked >= last.max(-1).values - 0.1).all())
        seq = torch.cat([seq, tokens[:, 0, t:t + 1].long()], 1)
