"""The loop of drafted generation without a GPU: models whose logits are a table of the last token, and the
verification by its definition in place of the library's."""

import pytest

from distilled_modal_ssm_amd import binding as hb
from distilled_modal_ssm_amd import hybrid


class _Verify:
    """DraftVerify on the host; probabilities that are none count as 0, and rows without any draw -1."""

    def __init__(self, batch, drafts, vocab, device=None):
        self.T = drafts

    def verify(self, p, tokens, u, q=None):
        import torch
        clean = lambda x: torch.where(torch.isfinite(x) & (x > 0), x, 0.0 * torch.ones_like(x)).double()  # noqa: E731
        p, q = clean(p), None if q is None else clean(q)
        out, counts = torch.full((p.shape[0], self.T + 1), -1, dtype=torch.int32), []
        for b in range(p.shape[0]):
            n = 0
            while n < self.T and 0 <= (x := int(tokens[b, n])) and float(u[b, n]) * float(q[b, n, x]) < float(p[b, n, x]):
                out[b, n] = x
                n += 1
            w = p[b, n]
            if n < self.T:
                left = (w - q[b, n]).clamp(min=0)
                w = left if float(left.sum()) > 0 else w
            over = torch.nonzero(w.cumsum(0) > float(u[b, self.T]) * float(w.sum()))
            out[b, n] = int(over[0]) if len(over) else -1
            counts.append(n)
        return out, torch.tensor(counts, dtype=torch.int32)


class _Table(hybrid.HybridLM):
    """Its state is a count of the tokens read; logits of a row: table[last token], or change(count, logits)."""

    def __init__(self, table, change=None):
        import torch
        super().__init__([], torch.zeros(table.shape[0], 4), None, device="cpu")
        self.table, self.change = table, change

    def _logits(self, count, tokens):
        logits = self.table[tokens.long()].clone()
        return self.change(count, logits) if self.change else logits

    def _operators(self, rows):
        return []

    def prefill(self, tokens, last=False):
        import torch
        count = torch.full((tokens.shape[0],), tokens.shape[1])
        return self._logits(count, tokens[:, -1]), [count]

    def _step(self, ops, states, tokens):
        states[0] += 1
        return self._logits(states[0], tokens)

    def _extend(self, ops, states, tokens, head=True):
        import torch
        logits = [self._logits(states[0] + 1 + t, tokens[:, t]) for t in range(tokens.shape[1])]
        return torch.stack(logits, 1), None

    def _commit(self, ops, states, seen, lengths):
        states[0] += lengths


class _On:
    """Stands in for the binding's: the devices that are current, one inside the other."""

    current = []

    def __init__(self, device, stream):
        self.device = device

    def __enter__(self):
        self.current.append(self.device)

    def __exit__(self, *exc):
        self.current.pop()


@pytest.fixture
def verified(monkeypatch):
    monkeypatch.setattr(hybrid, "DraftVerify", _Verify)
    monkeypatch.setattr(hb, "_On", _On)


def _models(torch, change=None, draft_change=None, V=40):
    g = torch.Generator().manual_seed(3)
    return _Table(4 * torch.randn(V, V, generator=g), change), _Table(4 * torch.randn(V, V, generator=g), draft_change)


def _greedy(table, prompts, steps):
    out, x = [], prompts[:, -1]
    for _ in range(steps):
        x = table[x].argmax(-1)
        out.append(x)
    return out


@pytest.mark.parametrize("temperature", [1e-4, 1e-30, 1e-38, 1e-42, 5e-324])
def test_any_temperature_above_zero(verified, temperature):
    """The coldest ones are greedy: no logit leaves float32's range on the way."""
    import torch
    model, draft = _models(torch)
    prompts = torch.arange(12).view(6, 2)
    tokens, rate = model.generate_drafted(prompts, draft, 9, drafts=3, temperature=temperature)
    assert torch.equal(tokens.long(), torch.stack(_greedy(model.table, prompts, 9), 1)) and 0 <= rate < 1


@pytest.mark.parametrize("at", [2, 3, 5, 10])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_logits_that_give_no_probabilities(verified, at, value):
    """Behind ``at`` tokens one row has none: an error, not tokens of -1, once they are to be returned."""
    import torch

    def change(count, logits):
        logits[3][count[3] == at] = value
        return logits

    model, draft = _models(torch, change)
    prompts = torch.arange(12).view(6, 2)
    with pytest.raises(ValueError):
        model.generate_drafted(prompts, draft, 9, drafts=3, temperature=1e-4)
    if at > 2:  # read, if at all, for tokens behind the last one asked for
        tokens, _ = model.generate_drafted(prompts, draft, at - 2, drafts=3, temperature=1e-4)
        assert torch.equal(tokens.long(), torch.stack(_greedy(model.table, prompts, at - 2), 1))


def test_a_draft_without_probabilities_is_refused(verified):
    """The target's tokens do not depend on it."""
    import torch

    def change(count, logits):
        logits[2][count[2] >= 4] = float("nan")
        return logits

    model, draft = _models(torch, None, change)
    prompts = torch.arange(12).view(6, 2)
    tokens, _ = model.generate_drafted(prompts, draft, 9, drafts=3, temperature=1e-4)
    assert torch.equal(tokens.long(), torch.stack(_greedy(model.table, prompts, 9), 1))


@pytest.mark.parametrize("call", ["prefill", "generate", "generate_drafted"])
def test_the_models_device_is_current(monkeypatch, call):
    """At the library's calls, whichever device is current for the caller."""
    import torch

    class Reached(Exception):
        pass

    def library(*args):
        assert _On.current and all(d == model.device for d in _On.current)
        raise Reached

    monkeypatch.setattr(hb, "_On", _On)
    monkeypatch.setattr(hybrid, "DraftVerify", _Verify)
    monkeypatch.setattr(hb, "hyena_dense_bf16", library)
    # (the prompt's logits would make it current for themselves alone)
    inner = hybrid.HybridLM.prefill
    monkeypatch.setattr(hybrid.HybridLM, "prefill", getattr(inner, "__wrapped__", inner) if call != "prefill" else inner)
    model = hybrid.HybridLM([], torch.zeros(50, 64), torch.zeros(50, 64), device="cpu")
    prompts = torch.zeros(2, 3, dtype=torch.int64)
    args = {"prefill": (prompts,), "generate": (prompts, 2, 3), "generate_drafted": (prompts, model, 3)}
    with pytest.raises(Reached):
        getattr(model, call)(*args[call])


def test_a_draft_on_another_device_is_refused(verified):
    import torch
    model, draft = _models(torch)
    draft.device = torch.device("meta")
    with pytest.raises(ValueError):
        model.generate_drafted(torch.zeros(1, 2, dtype=torch.int64), draft, 3)
