"""Verification of drafted tokens over the C ABI, on torch tensors.

A drafting model proposes a few tokens a sequence, the target model reads them
all in one pass, and this decides from both models' probabilities and given
random numbers which are kept and what comes behind them, so that the tokens are
distributed as the target's own.
"""

from __future__ import annotations

from . import binding as hb


class DraftVerify:
    """Sizes and workspace of a verification, and its call.

    batch sequences of up to ``drafts`` drafted tokens each, over ``vocab``
    tokens.  drafts = 0 draws one token a sequence.
    """

    def __init__(self, batch: int, drafts: int, vocab: int, device="cuda"):
        import torch
        self.torch = torch
        self.device = torch.empty(0, device=device).device  # with its index
        self.B, self.T, self.V = int(batch), int(drafts), int(vocab)
        self.ws_bytes = hb.hyena_draft_verify_workspace(self.B, self.T, self.V)
        self._ws = hb._Scratch()  # a captured graph has its own
        self._verify = hb.load().hyena_draft_verify
        self._p_shape, self._q_shape = (self.B, self.T + 1, self.V), (self.B, self.T, self.V)
        self._x_shape, self._u_shape, self._rows = (self.B, self.T), (self.B, self.T + 1), (self.B,)

    def _probs(self, name, t, shape, dtype):
        """Row stride of probabilities [B][places][V]."""
        if t.dtype != dtype or t.shape != shape or t.device != self.device:
            raise ValueError(f"{name}: need {dtype} {shape} on {self.device}, got {t.dtype} {tuple(t.shape)} on "
                             f"{t.device}")
        ld = self.V if t.is_contiguous() else hb._row_stride(t, ())
        if ld < self.V:
            raise ValueError(f"{name}: rows overlap")
        return ld

    def verify(self, p, tokens, u, q=None, lengths=None, out=None, stream=None):
        """(tokens int32 [B][drafts + 1], accepted int32 [B]): the kept drafts, one drawn token, then
        -1; and how many drafts were kept.

        p [B][drafts + 1][V]: the target's probabilities at each drafted token's
        place and behind the last, float32 or bfloat16.  tokens int32
        [B][drafts].  u float32 [B][drafts + 1] in [0, 1): one a draft, the last
        for the drawn token.  q [B][drafts][V]: the drafting model's
        probabilities, of p's type, or None where it drafts without chance.
        lengths int32 [B]: drafted tokens of each sequence.
        """
        torch, dtype = self.torch, p.dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"p: need float32 or bfloat16, got {dtype}")
        ld_p = self._probs("p", p, self._p_shape, dtype)
        ld_q = 0 if q is None else self._probs("q", q, self._q_shape, dtype)
        hb._expect("tokens", tokens, torch.int32, self._x_shape, self.device)
        hb._expect("u", u, torch.float32, self._u_shape, self.device)
        if lengths is not None:
            hb._expect("lengths", lengths, torch.int32, self._rows, self.device)
        if out is not None:
            hb._expect("out tokens", out[0], torch.int32, self._u_shape, self.device)
            hb._expect("out accepted", out[1], torch.int32, self._rows, self.device)
        return hb._call(self._run, self.device, stream, p, ld_p, q, ld_q, tokens, lengths, u, out)

    def _run(self, p, ld_p, q, ld_q, tokens, lengths, u, out, stream):
        torch = self.torch
        if out is None:
            out = (torch.empty(self._u_shape, dtype=torch.int32, device=self.device),
                   torch.empty(self._rows, dtype=torch.int32, device=self.device))
        with self._ws.order(stream):
            ws = hb._scratch(self._ws, self.ws_bytes, stream, self.device)
            # (straight to the C entry point: a step's call counts in microseconds)
            hb._check(self._verify(self.B, self.T, self.V, hb.HM_BF16 if p.dtype == torch.bfloat16 else hb.HM_F32,
                                   p.data_ptr(), ld_p, None if q is None else q.data_ptr(), ld_q, tokens.data_ptr(),
                                   None if lengths is None else lengths.data_ptr(), u.data_ptr(), out[0].data_ptr(),
                                   out[1].data_ptr(), ws.data_ptr(), self.ws_bytes, stream), "hyena_draft_verify")
        return out
