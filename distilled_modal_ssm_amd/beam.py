"""Beam search over the C ABI, on torch tensors: the choice of each group's best
continuations, and the move of the layers' states to where their beams went.

A step of a search:
    scores, tokens, parents, finished = beam.select(logits, scores, finished)
    beam.reorder(parents, states)          # modal states, deferred u_prev and rho, ...
Linear-attention states need no reorder where the next decode step is given the
parents' rows (``beam.rows(parents)``).
"""

from __future__ import annotations

from . import binding as hb


class BeamSearch:
    """Sizes of a search and its workspace, and its calls.

    groups searches of ``beams`` beams each over ``vocab`` tokens; ``select``
    continuations are kept of each (``beams`` by default; a program that holds
    ended sequences apart keeps more and picks from them).  end_token: the token
    that ends a sequence, None for none.
    """

    def __init__(self, groups: int, beams: int, vocab: int, select=None, end_token=None, device="cuda"):
        import torch
        self.torch = torch
        self.device = torch.empty(0, device=device).device  # with its index
        self.groups, self.beams, self.vocab = int(groups), int(beams), int(vocab)
        self.n = self.beams if select is None else int(select)
        self.end_token = -1 if end_token is None else int(end_token)
        self.ws_bytes = hb.hyena_beam_select_workspace(self.groups, self.beams, self.vocab, self.n)
        self._ws = {}  # scratch memory of each stream; a captured graph has its own
        self._select = hb.load().hyena_beam_select
        # outputs are made like these: scores, tokens and parents in one allocation
        self._like = (torch.empty((3, self.groups, self.n), dtype=torch.int32, device=self.device),
                      torch.empty((self.groups, self.n), dtype=torch.uint8, device=self.device))
        self._logits_shape, self._beams_shape = (self.groups * self.beams, self.vocab), (self.groups, self.beams)

    def first_scores(self):
        """Scores of a search's start: one live beam in each group."""
        s = self.torch.full((self.groups, self.beams), float("-inf"), dtype=self.torch.float32, device=self.device)
        s[:, 0] = 0.0
        return s

    def select(self, logits, scores, finished=None, out=None, stream=None):
        """The best continuations (scores float32, tokens int32, parents int32, finished uint8), each
        [groups][select], best first.

        logits: [groups * beams][vocab] float32 or bfloat16, unit element stride;
        scores: float32 [groups][beams]; finished: uint8 [groups][beams] or None.
        out: the four tensors to write, instead of new ones.
        """
        torch, (rows, V) = self.torch, self._logits_shape
        dtype = logits.dtype
        if dtype not in (torch.float32, torch.bfloat16) or logits.shape != self._logits_shape \
                or logits.device != self.device or (V > 1 and logits.stride(1) != 1):
            raise ValueError(f"logits: need float32 or bfloat16 {self._logits_shape} rows on {self.device}, got {dtype} "
                             f"{tuple(logits.shape)} on {logits.device}")
        hb._expect("scores", scores, torch.float32, self._beams_shape, self.device)
        if finished is not None:
            hb._expect("finished", finished, torch.uint8, self._beams_shape, self.device)
        with hb._On(self.device, stream) as stream:
            if out is None:
                s, tokens, parents = torch.empty_like(self._like[0]).unbind(0)
                out = (s.view(torch.float32), tokens, parents, torch.empty_like(self._like[1]))
            else:
                for name, x, t in zip(("scores", "tokens", "parents", "finished"), out,
                                      (torch.float32, torch.int32, torch.int32, torch.uint8)):
                    hb._expect("out " + name, x, t, (self.groups, self.n), self.device)
            ws = hb._scratch(self._ws, self.ws_bytes, stream, self.device)
            # (straight to the C entry point: a step's call counts in microseconds)
            hb._check(self._select(self.groups, self.beams, V, self.n,
                                   hb.HM_BF16 if dtype == torch.bfloat16 else hb.HM_F32, logits.data_ptr(),
                                   logits.stride(0) if rows > 1 else V, scores.data_ptr(),
                                   None if finished is None else finished.data_ptr(), self.end_token,
                                   out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                                   ws.data_ptr(), self.ws_bytes, stream), "hyena_beam_select")
        return out

    def rows(self, parents):
        """parents [groups][beams] in the group -> rows [groups * beams] of the whole batch (int32)."""
        torch = self.torch
        base = torch.arange(0, self.groups * self.beams, self.beams, dtype=torch.int32, device=parents.device)
        return (parents + base[:, None]).reshape(-1)

    def reorder(self, parents, states, stream=None):
        """Moves rows of every state in place: row (g, k) <- old row (g, parents[g][k]).

        parents: int32 [groups][beams]; states: contiguous tensors whose first
        dimension is the groups * beams batch rows.
        """
        hb._expect("parents", parents, self.torch.int32, (self.groups, self.beams), self.device)
        rows = self.groups * self.beams
        sizes = []
        for i, s in enumerate(states):
            if s.dim() < 1 or s.shape[0] != rows or s.device != self.device or not s.is_contiguous():
                raise ValueError(f"states[{i}]: need a contiguous tensor of {rows} rows on {self.device}, got "
                                 f"{tuple(s.shape)} on {s.device}")
            sizes.append(s.numel() // rows * s.element_size() if rows else 0)
        with hb._On(self.device, stream) as stream:
            hb.hyena_beam_reorder(self.groups, self.beams, parents, states, sizes, stream)
