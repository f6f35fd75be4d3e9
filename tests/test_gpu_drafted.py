"""Drafted generation over a hybrid model (modal Hyena, linear attention, gated recurrence), end to
end: the gated recurrence, the 8-bit products and the verification run together as they are used.

Tolerances.  A pass over several tokens and a step a token round the same values to
bfloat16 at the same places but sum in another order, so an activation may land on
the neighbouring bfloat16 value (2^-8 of it); with L layers of two products,
sign-random, a logit of size up to 12 moves by some 12 * 2^-8 * sqrt(2 L) / 3 = 0.05
for L = 4, and a state by 2^-8 sqrt(2 L) = 0.011 of its norm.  Twice these are
allowed.  A state that went on with a refused draft moves by a good part of itself.
"""

import os
import sys

import pytest

from _gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _model(torch, kinds, width, vocab, seed=0, like=None):
    from drafted_generate import random_model
    return random_model(torch, kinds, width, vocab, heads=4, modes=8, seed=seed, like=like)


ALL = ("gated", "hyena", "attention", "gated")


@pytest.mark.parametrize("eight", [False, True])
def test_states_behind_the_kept_tokens(eight):
    torch = require_gpu()
    log(f"states {eight}")
    model = _model(torch, ALL, 128, 300)
    model = model.quantized() if eight else model
    B, n = 5, 6
    g = torch.Generator().manual_seed(1)
    prompts, more = torch.randint(0, 300, (B, 20), generator=g).cuda(), torch.randint(0, 300, (B, n), generator=g).cuda()
    lengths = torch.tensor([1, 6, 3, 2, 5], dtype=torch.int32).cuda()
    _, states = model.prefill(prompts)
    before = [s.clone() for s in states]
    ops = model._operators(B)
    logits, seen = model._extend(ops, states, more)
    assert all(torch.equal(a, b) for a, b in zip(states, before))
    model._commit(ops, states, seen, lengths)
    want, step = [s.clone() for s in before], [s.clone() for s in before]
    for t in range(n):
        one = model._step(ops, step, more[:, t])
        assert float((one.float() - logits[:, t].float()).abs().max()) <= (0.4 if eight else 0.1)
        for w, s in zip(want, step):
            w[lengths == t + 1] = s[lengths == t + 1]
    for got, w, b in zip(states, want, before):
        for r in range(B):
            assert float((got[r] - w[r]).norm()) <= (0.1 if eight else 0.022) * float(w[r].norm())
            assert float((got[r] - b[r]).norm()) > 0.1 * float(w[r].norm())


@pytest.mark.parametrize("drafts", [1, 4, 9])
def test_cold_drafts_are_greedy(drafts):
    """At a temperature near 0 every token is the likeliest behind those before it, whoever drafted it."""
    torch = require_gpu()
    log(f"cold {drafts}")
    model = _model(torch, ALL, 128, 400)
    draft = _model(torch, ("gated",), 64, 400, like=model)
    prompts = torch.randint(0, 400, (6, 33), generator=torch.Generator().manual_seed(2)).cuda()
    steps = 11
    tokens, rate = model.generate_drafted(prompts, draft, steps, drafts=drafts, temperature=1e-4)
    assert tokens.shape == (6, steps) and 0 <= rate <= 1
    logits, _ = model.prefill(torch.cat([prompts, tokens.long()], 1))
    logits = logits.view(6, 33 + steps, 400).float()[:, 32:-1]
    picked = logits.gather(2, tokens[..., None].long())[..., 0]
    assert float((logits.max(-1).values - picked).max()) <= 0.1
    # its own drafts are kept, but where two tokens are nearly as likely
    again, rate = model.generate_drafted(prompts, model, steps, drafts=drafts, temperature=1e-4)
    assert rate > 0.8


def test_tokens_are_distributed_as_without_drafts():
    """The second and third token of 8192 continuations of one prompt against their exact distribution:
    every frequency within 5 standard deviations (and the tolerance of the logits, 10 % of it)."""
    torch = require_gpu()
    log("distribution")
    V, B = 64, 8192
    model = _model(torch, ("gated", "attention"), 64, V, seed=3)
    draft = _model(torch, ("gated",), 64, V, seed=4)
    prompt = torch.randint(0, V, (1, 9), generator=torch.Generator().manual_seed(5)).cuda()
    heat = 6.0  # flat enough that every token counts
    p1 = torch.softmax(model.prefill(prompt, last=True)[0].double() / heat, -1)[0]
    firsts = torch.cat([prompt.expand(V, 9), torch.arange(V, device="cuda")[:, None]], 1)
    p2 = torch.softmax(model.prefill(firsts, last=True)[0].double() / heat, -1)  # [first][second]
    pairs = torch.cat([firsts.repeat_interleave(V, 0), torch.arange(V, device="cuda").repeat(V)[:, None]], 1)
    p3 = torch.softmax(model.prefill(pairs, last=True)[0].double() / heat, -1).view(V, V, V)
    second = p1 @ p2
    third = torch.einsum("a,ab,abc->c", p1.cpu(), p2.cpu(), p3.cpu()).cuda()
    g = torch.Generator(device="cuda").manual_seed(6)
    tokens, rate = model.generate_drafted(prompt.expand(B, 9), draft, 3, drafts=2, temperature=heat, generator=g)
    assert 0.2 < rate < 0.999  # some kept and some refused
    for t, want in ((0, p1), (1, second), (2, third)):
        freq = torch.bincount(tokens[:, t].long(), minlength=V).double() / B
        dev = 5 * (want * (1 - want) / B).sqrt() + 0.1 * want
        assert bool(((freq - want).abs() <= dev).all()), (t, float(((freq - want).abs() / dev).max()))


def test_beams_of_a_gated_model():
    """Beam search moves the gated states as it does the others: sequences score as prompts."""
    torch = require_gpu()
    log("gated beams")
    model = _model(torch, ("gated", "attention", "gated"), 128, 500, seed=7)
    G, K, L, steps = 2, 4, 21, 8
    prompts = torch.randint(0, 500, (G, L), generator=torch.Generator().manual_seed(L)).cuda()
    tokens, scores = model.generate(prompts, K, steps)
    whole = torch.cat([prompts.repeat_interleave(K, 0), tokens.reshape(G * K, steps).long()], 1)
    logits, _ = model.prefill(whole)
    logp = torch.log_softmax(logits.view(G * K, L + steps, -1).double(), -1)[:, L - 1:-1]
    want = logp.gather(2, tokens.reshape(G * K, steps, 1).long())[..., 0].sum(-1)
    assert float((scores.reshape(-1) - want).abs().max()) <= 0.1 * steps


def test_quantized_model_answers_alike():
    """A product in 8 bits is off by some 2^-7 / sqrt(12) * 3 of its terms (rows whose largest value is three
    times their mean size), twice: 1 % of a layer's output, and 5 % behind four layers of two and a head."""
    torch = require_gpu()
    log("quantized")
    model = _model(torch, ALL, 128, 500)
    prompts = torch.randint(0, 500, (3, 40), generator=torch.Generator().manual_seed(1)).cuda()
    a, b = model.prefill(prompts)[0].float(), model.quantized().prefill(prompts)[0].float()
    assert 0 < float((a - b).norm() / a.norm()) < 0.15


def test_refusals_and_the_example():
    torch = require_gpu()
    model, other = _model(torch, ("gated",), 64, 100), _model(torch, ("gated",), 64, 128)
    prompts = torch.zeros((1, 4), dtype=torch.int64, device="cuda")
    for kw in (dict(draft=other), dict(draft=model, drafts=0), dict(draft=model, temperature=0.0), dict(draft=model, steps=0)):
        with pytest.raises(ValueError):
            model.generate_drafted(prompts, **{"steps": 3, **kw})
    import drafted_generate
    drafted_generate.main(["--layers", "2", "--width", "64", "--vocab", "200", "--prompt", "20", "--steps", "5",
                           "--batch", "2"])


@pytest.mark.parametrize("temperature", [1e-30, 1e-38, 1e-300])
def test_the_coldest_drafts_are_greedy(temperature):
    """As at 1e-4: no logit leaves float32's range."""
    torch = require_gpu()
    log(f"coldest {temperature}")
    model = _model(torch, ALL, 128, 400)
    draft = _model(torch, ("gated",), 64, 400, like=model)
    prompts = torch.randint(0, 400, (6, 33), generator=torch.Generator().manual_seed(2)).cuda()
    tokens, _ = model.generate_drafted(prompts, draft, 7, drafts=3, temperature=temperature)
    logits, _ = model.prefill(torch.cat([prompts, tokens.long()], 1))
    logits = logits.view(6, 40, 400).float()[:, 32:-1]
    picked = logits.gather(2, tokens[..., None].long())[..., 0]
    assert float((logits.max(-1).values - picked).max()) <= 0.1


@pytest.mark.parametrize("eight", [False, True])
def test_weights_that_are_not_finite_raise(eight):
    torch = require_gpu()
    log(f"not finite {eight}")
    model = _model(torch, ALL, 128, 400)
    prompts = torch.randint(0, 400, (3, 9), generator=torch.Generator().manual_seed(2)).cuda()
    model.embedding = model.embedding.clone()
    model.embedding[prompts[1, -1]] = float("nan")
    model = model.quantized() if eight else model
    draft = _model(torch, ("gated",), 64, 400)
    with pytest.raises(ValueError):
        model.generate_drafted(prompts, draft, 5, drafts=3)
