"""A hybrid language model over the C ABI, generating by beam search.

Every layer: in_proj (D -> 3D) of the input with each row scaled by its inverse
RMS -> [q|k|v] through the layer's operator -> out_proj (D -> D).  The operator
is the modal Hyena operator or linear attention with a decay; both keep a state
of constant size a row.  Token embeddings feed the first layer, a head (D ->
vocab) reads the last.  Every computation is a library call; torch provides
memory, views, streams and the lookup of embeddings.

A generated token of a search of K beams a prompt:
    logits -> select -> (scores, tokens, parents, finished)
    modal states: moved to their beams in place, all layers in one call;
    linear-attention states: read through the parents' rows by the next step
    itself, from one of two buffers into the other.
"""

from __future__ import annotations

from . import binding as hb
from .beam import BeamSearch
from .linear_attention import LinearAttention

RMS_EPS = 1e-6


class HybridLM:
    """layers: a list of ("hyena", params, W_in [3D][D], W_out [D][D]) with
    ModalParams-like tables (poles, residues, skip), and ("attention", log_decay
    [heads], W_in, W_out).  embedding [vocab][D], head [vocab][D]; weights are
    bfloat16 tensors on ``device``, D a multiple of 64."""

    def __init__(self, layers, embedding, head, device="cuda"):
        import torch
        self.torch = torch
        self.device = torch.device(device)
        self.layers = layers
        self.embedding, self.head = embedding, head
        self.vocab, self.D = int(embedding.shape[0]), int(embedding.shape[1])

    def _operators(self, rows: int):
        """The layers' operators for a batch of ``rows``."""
        ops = []
        for kind, p, _, _ in self.layers:
            if kind == "hyena":
                ops.append(hb.ModalHyena(p.poles, p.residues, p.skip, rows, self.D, "bf16", device=self.device))
            else:
                H = int(p.shape[0])
                ops.append(LinearAttention(rows, H, self.D // H, self.D // H, "bf16", device=self.device))
        return ops

    def _dense(self, x, w, out, rms=False):
        M, K = x.shape
        if rms:
            hb.hyena_dense_rms_bf16(M, w.shape[0], K, x, x.stride(0), w, w.stride(0), RMS_EPS, out, out.stride(0))
        else:
            hb.hyena_dense_bf16(M, w.shape[0], K, x, x.stride(0), w, w.stride(0), None, out, out.stride(0))
        return out

    def _new(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.bfloat16, device=self.device)

    def prefill(self, tokens, last=False):
        """tokens [B][L] -> (logits [B * L][vocab], or [B][vocab] of each prompt's ``last`` position
        alone, and the layers' states)."""
        B, L = tokens.shape
        D = self.D
        x = self.embedding[tokens.long()].reshape(B * L, D)
        states = []
        for op, (kind, p, w_in, w_out) in zip(self._operators(B), self.layers):
            q, k, v = self._dense(x, w_in, self._new(B * L, 3 * D), rms=True).view(B, L, 3, D).unbind(2)
            y, state = op.prefill(q, k, v) if kind == "hyena" else op.prefill(q, k, v, p)
            states.append(state)
            x = self._dense(y.view(B * L, D), w_out, self._new(B * L, D))
        if last:
            x = x.view(B, L, D)[:, -1].contiguous()
        return self._dense(x, self.head, self._new(x.shape[0], self.vocab)), states

    def generate(self, prompts, beams: int, steps: int, end_token=None):
        """The best ``beams`` continuations of every prompt [G][L]: (tokens [G][beams][steps],
        scores [G][beams]), best first.  Past its end a sequence repeats end_token."""
        torch, D = self.torch, self.D
        G = prompts.shape[0]
        rows = G * beams
        logits, states = self.prefill(prompts, last=True)
        logits = logits.repeat_interleave(beams, 0)
        states = [s.repeat_interleave(beams, 0) for s in states]
        other = [torch.empty_like(s) if kind == "attention" else None for s, (kind, *_) in zip(states, self.layers)]
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
                    op.decode_step(q, k, v, states[i], p, y=y, rows=source, state_out=other[i])
                    states[i], other[i] = other[i], states[i]
                self._dense(y, w_out, x)
            logits = self._dense(x, self.head, self._new(rows, self.vocab))
        # back from the last beams to their first tokens
        out, at = [], torch.arange(beams, device=self.device).expand(G, beams)
        for tokens, parents in reversed(history):
            out.append(tokens.gather(1, at))
            at = parents.long().gather(1, at)
        return torch.stack(out[::-1], -1), scores
