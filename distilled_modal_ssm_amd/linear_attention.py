"""Linear attention with a decay over the C ABI, on torch tensors.

Per batch row and head, with a float32 state S [key_dim][value_dim]:
    S_t = exp(a_t) S_{t-1} + k_t v_t^T,      y_t = scale S_t^T q_t.
The matrix-state layer that hybrid stacks put beside the modal Hyena operator
(the Telegram digest's post on state-space duality, the Based blog repost): the
same two modes, a prompt with its end state and one step a token.
"""

from __future__ import annotations

import ctypes

from . import binding as hb


class LinearAttention:
    """One layer's sizes and workspace, and its calls.

    act: "f32" or "bf16", the type of q, k, v and y.  q, k and v may have fewer
    heads than there are states: head h reads head h * q_heads // heads.
    scale: key_dim ** -0.5 by default.
    """

    def __init__(self, batch: int, heads: int, key_dim: int, value_dim: int, act: str, q_heads=None, k_heads=None,
                 v_heads=None, scale=None, device="cuda"):
        import torch
        if act not in ("f32", "bf16"):
            raise ValueError(f"unknown activation type {act!r}")
        self.torch = torch
        self.device = torch.empty(0, device=device).device  # with its index
        self.B, self.H, self.dk, self.dv = int(batch), int(heads), int(key_dim), int(value_dim)
        self.q_heads, self.k_heads, self.v_heads = (int(n) if n else self.H for n in (q_heads, k_heads, v_heads))
        self.tdtype = torch.bfloat16 if act == "bf16" else torch.float32
        self.scale = self.dk ** -0.5 if scale is None else float(scale)
        self.desc = hb.make_linattn_desc(self.B, self.H, self.dk, self.dv, hb.HM_BF16 if act == "bf16" else hb.HM_F32,
                                         self.scale, self.q_heads, self.k_heads, self.v_heads)
        hb.hyena_linattn_prefill_workspace(self.desc, 0)  # raises for sizes that the library refuses
        self._ws = {}  # scratch memory of each stream; a captured graph has its own
        self._state_shape = (self.B, self.H, self.dk, self.dv)
        self._token_shapes = ((self.B, self.q_heads * self.dk), (self.B, self.k_heads * self.dk),
                              (self.B, self.v_heads * self.dv), (self.B, self.H * self.dv))
        self._token, self._desc_ref = hb.load().hyena_linattn_decode_step, ctypes.byref(self.desc)

    def new_state(self):
        return self.torch.zeros((self.B, self.H, self.dk, self.dv), dtype=self.torch.float32, device=self.device)

    def _workspace(self, L, stream):
        n = hb.hyena_linattn_prefill_workspace(self.desc, L)
        if n == 0:
            return None, 0
        return hb._scratch(self._ws, n, stream, self.device), n

    def _rows(self, name, t, shape, dtype):
        """Row stride of rows [..][width] of this shape, row (b, t) at (b * L + t) * stride."""
        if t.dtype != dtype or t.shape != shape or t.device != self.device:
            raise ValueError(f"{name}: need {dtype} {shape} on {self.device}, got {t.dtype} {tuple(t.shape)} on "
                             f"{t.device}")
        if t.is_contiguous():
            return shape[-1]
        if len(shape) == 3:
            return hb._row_stride(t, ())
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: rows need unit element stride")
        return t.stride(0)

    def _decay(self, a, lead):
        """Row stride of a log decay: 0 for one a head."""
        if a is None:
            return 0
        if a.dim() == 1:
            hb._expect("log_decay", a, self.torch.float32, (self.H,), self.device)
            return 0
        return self._rows("log_decay", a, (*lead, self.H), self.torch.float32)

    def _state(self, name, s):
        hb._expect(name, s, self.torch.float32, self._state_shape, self.device)

    def prefill(self, q, k, v, log_decay=None, lengths=None, y=None, state_in=None, state_out=None, stream=None):
        """A prompt of L tokens.  Returns (y, state after each row's last token).

        q [B][L][q_heads * key_dim], k, v: views with unit element stride and batch
        rows one after the other.  log_decay: float32 [heads] or [B][L][heads]
        (<= 0), or None for no decay.  lengths: int32 [B], tokens of each row
        (later ones are not read, their y is 0).  state_out may be state_in.
        """
        L = int(q.shape[1]) if q.dim() == 3 else -1
        lead, dt = (self.B, L), self.tdtype
        ld_q = self._rows("q", q, (*lead, self.q_heads * self.dk), dt)
        ld_k = self._rows("k", k, (*lead, self.k_heads * self.dk), dt)
        ld_v = self._rows("v", v, (*lead, self.v_heads * self.dv), dt)
        ld_a = self._decay(log_decay, lead)
        if lengths is not None:
            hb._expect("lengths", lengths, self.torch.int32, (self.B,), self.device)
        if state_in is not None:
            self._state("state_in", state_in)
        with hb._On(self.device, stream) as stream:
            if y is None:
                y = self.torch.empty((*lead, self.H * self.dv), dtype=dt, device=self.device)
            if state_out is None:
                state_out = self.torch.empty(self._state_shape, dtype=self.torch.float32, device=self.device)
            else:
                self._state("state_out", state_out)
            ws, n = self._workspace(L, stream)
            hb.hyena_linattn_prefill(self.desc, L, lengths, q, ld_q, k, ld_k, v, ld_v, log_decay, ld_a, y,
                                     self._rows("y", y, (*lead, self.H * self.dv), dt), state_in, state_out, ws, n,
                                     stream)
        return y, state_out

    def decode_step(self, q, k, v, state, log_decay=None, y=None, rows=None, state_out=None, stream=None):
        """One token for every batch row.  Returns y [B][heads * value_dim].

        q [B][q_heads * key_dim], k, v: rows with unit element stride.  log_decay:
        [heads] or [B][heads].  The state is updated in place, or read and written
        to ``state_out``; with ``rows`` (int32 [B]) batch row b continues row
        rows[b] of ``state``, and ``state_out`` must be another tensor.
        """
        dt = self.tdtype
        ld_q = self._rows("q", q, self._token_shapes[0], dt)
        ld_k = self._rows("k", k, self._token_shapes[1], dt)
        ld_v = self._rows("v", v, self._token_shapes[2], dt)
        ld_a = self._decay(log_decay, (self.B,))
        self._state("state", state)
        if rows is not None:
            hb._expect("rows", rows, self.torch.int32, (self.B,), self.device)
            if state_out is None:
                raise ValueError("rows need a state_out beside the state")
        if state_out is None:
            state_out = state
        else:
            self._state("state_out", state_out)
        with hb._On(self.device, stream) as stream:
            if y is None:
                y = self.torch.empty(self._token_shapes[3], dtype=dt, device=self.device)
            # (straight to the C entry point: a token's call counts in microseconds)
            hb._check(self._token(self._desc_ref, q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v,
                                  None if log_decay is None else log_decay.data_ptr(), ld_a, y.data_ptr(),
                                  self._rows("y", y, self._token_shapes[3], dt), state.data_ptr(),
                                  None if rows is None else rows.data_ptr(), state_out.data_ptr(), stream),
                      "hyena_linattn_decode_step")
        return y
