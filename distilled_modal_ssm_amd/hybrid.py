"""A hybrid language model over the C ABI, generating by beam search, or by
chance with another model's drafts.

Every layer: in_proj (D -> 3D) of the input with each row scaled by its inverse
RMS -> [q|k|v] through the layer's operator -> out_proj (D -> D).  The operator
is the modal Hyena operator, linear attention with a decay or the gated
recurrence (k its gate's logits); all keep a state of constant size a row.
Token embeddings feed the first layer, a head (D -> vocab) reads the last.
Projections are bfloat16, or in 8 bits (``quantized``).  Every computation is a
library call; torch provides memory, views, streams, the lookup of embeddings
and the softmax of drafted generation.

A generated token of a search of K beams a prompt:
    logits -> select -> (scores, tokens, parents, finished)
    modal states: moved to their beams in place, all layers in one call;
    linear-attention states: read through the parents' rows by the next step
    itself, from one of two buffers into the other; gated states likewise.

Drafted tokens of a sequence: a smaller model draws T tokens one by one, this one
reads the last token and those in one pass, and the verification keeps some and
draws one more.  Both models then take their states from before the drafts to
behind the kept ones: attention and gated layers run their operator again over
the pass's q, k and v with the kept lengths; modal layers, whose prompt form has
no lengths, step through the pass token by token and keep the state of each.
"""

from __future__ import annotations

import functools

from . import binding as hb
from .beam import BeamSearch
from .drafts import DraftVerify
from .int8 import Int8Dense
from .linear_attention import LinearAttention
from .recurrence import GatedRecurrence

RMS_EPS = 1e-6


def _on_device(method):
    """``method`` with the model's device current: the library works on the current device's memory."""
    @functools.wraps(method)
    def call(self, *args, **kw):
        with hb._On(self.device, None):
            return method(self, *args, **kw)
    return call


class HybridLM:
    """layers: a list of ("hyena", params, W_in [3D][D], W_out [D][D]) with
    ModalParams-like tables (poles, residues, skip), ("attention", log_decay
    [heads], W_in, W_out), and ("gated", input, W_in, W_out) with the gate's
    input factor ("convex", "norm" or "free").  embedding [vocab][D], head
    [vocab][D]; weights are bfloat16 tensors on ``device`` (W_in, W_out and head
    may be Int8Dense), D a multiple of 64."""

    def __init__(self, layers, embedding, head, device="cuda"):
        import torch
        self.torch = torch
        self.device = torch.empty(0, device=device).device  # with its index
        self.layers = layers
        self.embedding, self.head = embedding, head
        self.vocab, self.D = int(embedding.shape[0]), int(embedding.shape[1])

    def _operators(self, rows: int):
        """The layers' operators for a batch of ``rows``."""
        ops = []
        for kind, p, _, _ in self.layers:
            if kind == "hyena":
                ops.append(hb.ModalHyena(p.poles, p.residues, p.skip, rows, self.D, "bf16", device=self.device))
            elif kind == "gated":
                ops.append(GatedRecurrence(rows, self.D, "bf16", input=p, device=self.device))
            else:
                H = int(p.shape[0])
                ops.append(LinearAttention(rows, H, self.D // H, self.D // H, "bf16", device=self.device))
        return ops

    def quantized(self):
        """This model with its projections and its head in 8-bit integers."""
        eight = lambda w: w if isinstance(w, Int8Dense) else Int8Dense(w)  # noqa: E731
        layers = [(kind, p, eight(w_in), eight(w_out)) for kind, p, w_in, w_out in self.layers]
        return HybridLM(layers, self.embedding, eight(self.head), device=self.device)

    def _dense(self, x, w, out, rms=False):
        M, K = x.shape
        if isinstance(w, Int8Dense):
            w(x, out=out, rms_eps=RMS_EPS if rms else None)
        elif rms:
            hb.hyena_dense_rms_bf16(M, w.shape[0], K, x, x.stride(0), w, w.stride(0), RMS_EPS, out, out.stride(0))
        else:
            hb.hyena_dense_bf16(M, w.shape[0], K, x, x.stride(0), w, w.stride(0), None, out, out.stride(0))
        return out

    def _new(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.bfloat16, device=self.device)

    @_on_device
    def prefill(self, tokens, last=False):
        """tokens [B][L] -> (logits [B * L][vocab], or [B][vocab] of each prompt's ``last`` position
        alone, and the layers' states)."""
        B, L = tokens.shape
        D = self.D
        x = self.embedding[tokens.long()].reshape(B * L, D)
        states = []
        for op, (kind, p, w_in, w_out) in zip(self._operators(B), self.layers):
            q, k, v = self._dense(x, w_in, self._new(B * L, 3 * D), rms=True).view(B, L, 3, D).unbind(2)
            y, state = op.prefill(q, k, v, p) if kind == "attention" else op.prefill(q, k, v)
            states.append(state)
            x = self._dense(y.view(B * L, D), w_out, self._new(B * L, D))
        if last:
            x = x.view(B, L, D)[:, -1].contiguous()
        return self._dense(x, self.head, self._new(x.shape[0], self.vocab)), states

    @_on_device
    def generate(self, prompts, beams: int, steps: int, end_token=None):
        """The best ``beams`` continuations of every prompt [G][L]: (tokens [G][beams][steps],
        scores [G][beams]), best first.  Past its end a sequence repeats end_token."""
        torch, D = self.torch, self.D
        G = prompts.shape[0]
        rows = G * beams
        logits, states = self.prefill(prompts, last=True)
        logits = logits.repeat_interleave(beams, 0)
        states = [s.repeat_interleave(beams, 0) for s in states]
        other = [torch.empty_like(s) if kind != "hyena" else None for s, (kind, *_) in zip(states, self.layers)]
        modal = [s for s, (kind, *_) in zip(states, self.layers) if kind == "hyena"]
        ops = self._operators(rows)
        search = BeamSearch(G, beams, self.vocab, end_token=end_token, device=self.device)
        scores = search.first_scores()
        finished = torch.zeros((G, beams), dtype=torch.uint8, device=self.device) if end_token is not None else None
        qkv, y, x = self._new(rows, 3 * D), self._new(rows, D), self._new(rows, D)
        history = []
        for step in range(steps):
            scores, tokens, parents, ended = search.select(logits, scores, finished)
            finished = ended if end_token is not None else None
            history.append((tokens, parents))
            if step + 1 == steps:
                break
            search.reorder(parents, modal)
            source = search.rows(parents)
            x.copy_(self.embedding[tokens.view(-1).long()])
            for i, (op, (kind, p, w_in, w_out)) in enumerate(zip(ops, self.layers)):
                self._dense(x, w_in, qkv, rms=True)
                q, k, v = qkv[:, :D], qkv[:, D:2 * D], qkv[:, 2 * D:]
                if kind == "hyena":
                    op.decode_step(q, k, v, states[i], y=y)
                else:
                    args = (p,) if kind == "attention" else ()
                    op.decode_step(q, k, v, states[i], *args, y=y, rows=source, state_out=other[i])
                    states[i], other[i] = other[i], states[i]
                self._dense(y, w_out, x)
            logits = self._dense(x, self.head, self._new(rows, self.vocab))
        # back from the last beams to their first tokens
        out, at = [], torch.arange(beams, device=self.device).expand(G, beams)
        for tokens, parents in reversed(history):
            out.append(tokens.gather(1, at))
            at = parents.long().gather(1, at)
        return torch.stack(out[::-1], -1), scores

    def _step(self, ops, states, tokens):
        """One token a row: logits [B][vocab]; the states are updated in place."""
        D, B = self.D, tokens.shape[0]
        x = self.embedding[tokens.long()]
        for op, state, (kind, p, w_in, w_out) in zip(ops, states, self.layers):
            qkv = self._dense(x, w_in, self._new(B, 3 * D), rms=True)
            args = (p,) if kind == "attention" else ()
            y = op.decode_step(qkv[:, :D], qkv[:, D:2 * D], qkv[:, 2 * D:], state, *args)
            x = self._dense(y, w_out, self._new(B, D))
        return self._dense(x, self.head, self._new(B, self.vocab))

    def _extend(self, ops, states, tokens, head=True):
        """A few tokens a row behind the states, which stay: (logits [B][n][vocab] or None, what ``_commit`` needs)."""
        torch, D = self.torch, self.D
        B, n = tokens.shape
        x = self.embedding[tokens.long()].reshape(B * n, D)
        seen = []
        for op, state, (kind, p, w_in, w_out) in zip(ops, states, self.layers):
            q, k, v = self._dense(x, w_in, self._new(B * n, 3 * D), rms=True).view(B, n, 3, D).unbind(2)
            if kind == "hyena":
                after = torch.empty((n, *state.shape), dtype=state.dtype, device=self.device)
                y = self._new(B, n, D)
                for t in range(n):
                    after[t].copy_(state if t == 0 else after[t - 1])
                    op.decode_step(q[:, t], k[:, t], v[:, t], after[t], y=y[:, t])
                seen.append(after)
            else:
                y, _ = op.prefill(q, k, v, *((p,) if kind == "attention" else ()), state_in=state)
                seen.append((q, k, v))
            x = self._dense(y.view(B * n, D), w_out, self._new(B * n, D))
        logits = self._dense(x, self.head, self._new(B * n, self.vocab)).view(B, n, self.vocab) if head else None
        return logits, seen

    def _commit(self, ops, states, seen, lengths):
        """The states behind the first ``lengths`` (int32 [B], at least 1) tokens of an ``_extend``, in place."""
        for op, state, kept, (kind, p, *_) in zip(ops, states, seen, self.layers):
            if kind == "hyena":
                rows = self.torch.arange(state.shape[0], device=self.device)
                state.copy_(kept[lengths.long() - 1, rows])
            else:
                op.prefill(*kept, *((p,) if kind == "attention" else ()), lengths=lengths, state_in=state,
                           state_out=state)

    @_on_device
    def generate_drafted(self, prompts, draft, steps: int, drafts=4, temperature=1.0, generator=None):
        """``steps`` tokens drawn behind every prompt [B][L], distributed as this model's at the given
        temperature (one below 2^-126 counts as that), with the help of ``draft``, a HybridLM of the same
        vocabulary.

        Returns (tokens [B][steps], rate of drafted tokens that were kept).  Raises ValueError where this
        model's logits for one of them give no probabilities; a draft's that do not are refused.
        """
        torch, T = self.torch, int(drafts)
        if draft.vocab != self.vocab or draft.device != self.device:
            raise ValueError("the drafting model needs the same vocabulary and device")
        if T < 1 or steps < 1 or not temperature > 0:
            raise ValueError("need at least one draft and one step, and a temperature above 0")
        B = prompts.shape[0]
        cold = max(float(temperature), 2.0 ** -126)  # (1 / cold is a float32 too)

        def probs(logits):
            logits = logits.float()
            return torch.softmax((logits - logits.amax(-1, keepdim=True)) / cold, -1)  # (at most 0: none is infinite)

        rand = lambda n: torch.rand((B, n), generator=generator, device=self.device)  # noqa: E731
        one = DraftVerify(B, 0, self.vocab, device=self.device)
        several = DraftVerify(B, T, self.vocab, device=self.device)
        none = torch.empty((B, 0), dtype=torch.int32, device=self.device)
        draw = lambda p: one.verify(p.view(B, 1, self.vocab), none, rand(1))[0]  # noqa: E731
        logits, states = self.prefill(prompts, last=True)
        _, draft_states = draft.prefill(prompts, last=True)
        ops, draft_ops = self._operators(B), draft._operators(B)
        last = draw(probs(logits))
        # where each row's next tokens go; what is past `steps` is cut off at the end
        out = torch.zeros((B, steps + T + 1), dtype=torch.int32, device=self.device)
        out[:, :1] = last
        done = torch.ones((B, 1), dtype=torch.int64, device=self.device)
        place = torch.arange(T + 1, device=self.device)
        kept = asked = 0

        def progress(accepted):
            """The fewest tokens a row has, and drafts that were kept; what is returned holds no -1."""
            least, lowest, n = torch.stack([done.min(), out[:, :steps].min().long(), accepted.sum()]).tolist()
            if lowest < 0:
                raise ValueError("a prompt's logits give no probabilities (NaN or infinite)")
            return least, n

        least, _ = progress(done)
        while least < steps:
            trial, x, tokens, q = [s.clone() for s in draft_states], last, [last], []
            for _ in range(T):
                q.append(probs(draft._step(draft_ops, trial, x.view(B))))
                x = draw(q[-1])
                tokens.append(x)
            read = torch.cat(tokens, 1)
            logits, seen = self._extend(ops, states, read)
            _, draft_seen = draft._extend(draft_ops, draft_states, read, head=False)
            next_, accepted = several.verify(probs(logits), read[:, 1:].contiguous(), rand(T + 1), q=torch.stack(q, 1))
            lengths = accepted + 1
            self._commit(ops, states, seen, lengths)
            draft._commit(draft_ops, draft_states, draft_seen, lengths)
            last = next_.gather(1, accepted[:, None].long())
            # rows that have their steps write on behind them, in the same places again
            at = done.clamp(max=steps) + place
            out.scatter_(1, at, torch.where(place <= accepted[:, None], next_, out.gather(1, at)))
            done += lengths[:, None]
            least, n = progress(accepted)
            kept, asked = kept + n, asked + B * T
        return out[:, :steps], kept / max(asked, 1)
