"""Gated recurrence over the C ABI, on torch tensors.

Per batch row and channel, with a float32 state h:
    h_t = f_t h_{t-1} + i_t v_t,      y_t = q_t h_t      (y_t = h_t without q),
f = exp(g) or sigmoid(g), i = 1, 1 - f or sqrt(1 - f^2).  The vector-state layer
that hybrid stacks put beside the modal Hyena operator: a prompt with its end
state, one step a token, and the gradients of the prompt form.
"""

from __future__ import annotations

import ctypes

from . import binding as hb


class GatedRecurrence:
    """One layer's sizes and workspace, and its calls.

    act: "f32" or "bf16", the type of q, g, v, y and their gradients.
    gate: "sigmoid" (f of a logit) or "log" (f of a log decay, <= 0).
    input: "free", "convex" or "norm", the factor i of the inputs.
    """

    def __init__(self, batch: int, channels: int, act: str, gate="sigmoid", input="convex", device="cuda"):
        import torch
        if act not in ("f32", "bf16"):
            raise ValueError(f"unknown activation type {act!r}")
        if gate not in hb.GATES or input not in hb.GATE_INPUTS:
            raise ValueError(f"unknown gate {gate!r} or input {input!r}")
        self.torch = torch
        self.device = torch.empty(0, device=device).device  # with its index
        self.B, self.D = int(batch), int(channels)
        self.tdtype = torch.bfloat16 if act == "bf16" else torch.float32
        self.desc = hb.make_recurrence_desc(self.B, self.D, hb.HM_BF16 if act == "bf16" else hb.HM_F32, hb.GATES[gate],
                                            hb.GATE_INPUTS[input])
        hb.hyena_recurrence_workspace(self.desc, 0)  # raises for sizes that the library refuses
        self._ws = hb._Scratch()  # a captured graph has its own
        self._ws_bytes = {}  # of each length
        self._state_shape = (self.B, self.D)
        lib = hb.load()
        self._prompt, self._grads, self._token = (lib.hyena_recurrence_prefill, lib.hyena_recurrence_backward,
                                                  lib.hyena_recurrence_decode_step)
        self._desc_ref = ctypes.byref(self.desc)

    def new_state(self):
        return self.torch.zeros(self._state_shape, dtype=self.torch.float32, device=self.device)

    def new_chunk_states(self, L: int):
        """Memory for what a prompt of L tokens keeps for its backward pass."""
        n = -(-int(L) // hb.HM_RECURRENCE_CHUNK)
        return self.torch.empty((self.B, n, self.D), dtype=self.torch.float32, device=self.device)

    def _workspace(self, L, stream):
        n = self._ws_bytes.get(L)
        if n is None:
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            n = self._ws_bytes[L] = hb.hyena_recurrence_workspace(self.desc, L)
        return (hb._scratch(self._ws, n, stream, self.device), n) if n else (None, 0)

    def _rows(self, name, t, shape):
        """Row stride of rows [..][D] of this shape, row (b, t) at (b * L + t) * stride."""
        if t.dtype != self.tdtype or t.shape != shape or t.device != self.device:
            raise ValueError(f"{name}: need {self.tdtype} {tuple(shape)} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        strides = t.stride()
        ld = strides[-2]
        if len(shape) == 3 and ld >= self.D and strides == (shape[1] * ld, ld, 1):
            return ld
        if t.is_contiguous():
            return self.D
        if len(shape) == 3:
            ld = hb._row_stride(t, ())
        else:
            if self.D > 1 and strides[1] != 1:
                raise ValueError(f"{name}: rows need unit element stride")
            ld = ld if self.B > 1 else self.D
        if ld < self.D:
            raise ValueError(f"{name}: rows overlap")
        return ld

    def _inputs(self, q, g, v, lengths):
        """The rows' shape and the strides of q, g and v."""
        shape = (self.B, int(v.shape[1]) if v.dim() == 3 else -1, self.D)
        if lengths is not None:
            hb._expect("lengths", lengths, self.torch.int32, (self.B,), self.device)
        return shape, (0 if q is None else self._rows("q", q, shape), self._rows("g", g, shape),
                       self._rows("v", v, shape))

    def _f32(self, name, t, shape):
        hb._expect(name, t, self.torch.float32, shape, self.device)

    def prefill(self, q, g, v, lengths=None, y=None, state_in=None, state_out=None, chunk_states=None, stream=None):
        """A prompt of L tokens.  Returns (y, state after each row's last token).

        q (or None), g, v: [B][L][D] views with unit element stride and batch
        rows one after the other.  lengths: int32 [B], tokens of each row (later
        ones are not read, their y is 0).  state_out may be state_in; no other
        output may share memory with an input.
        chunk_states: memory as ``new_chunk_states`` gives it, which a backward
        pass reads.
        """
        shape, lds = self._inputs(q, g, v, lengths)
        if state_in is not None:
            self._f32("state_in", state_in, self._state_shape)
        if state_out is not None:
            self._f32("state_out", state_out, self._state_shape)
        if chunk_states is not None:
            self._f32("chunk_states", chunk_states, (self.B, -(-shape[1] // hb.HM_RECURRENCE_CHUNK), self.D))
        ld_y = self.D if y is None else self._rows("y", y, shape)
        return hb._call(self._run_prompt, self.device, stream, shape, q, g, v, lds, lengths, y, ld_y, state_in, state_out,
                        chunk_states)

    def _run_prompt(self, shape, q, g, v, lds, lengths, y, ld_y, state_in, state_out, chunk_states, stream):
        torch, L = self.torch, shape[1]
        if y is None:
            y = torch.empty(shape, dtype=self.tdtype, device=self.device)
        if state_out is None:
            state_out = torch.empty(self._state_shape, dtype=torch.float32, device=self.device)
        with self._ws.order(stream):
            ws, n = self._workspace(L, stream)
            # (straight to the C entry point: a few tokens' call counts in microseconds)
            hb._check(self._prompt(self._desc_ref, L, None if lengths is None else lengths.data_ptr(),
                                   None if q is None else q.data_ptr(), lds[0], g.data_ptr(), lds[1], v.data_ptr(), lds[2],
                                   y.data_ptr(), ld_y, None if state_in is None else state_in.data_ptr(),
                                   state_out.data_ptr(), None if chunk_states is None else chunk_states.data_ptr(),
                                   None if ws is None else ws.data_ptr(), n, stream), "hyena_recurrence_prefill")
        return y, state_out

    def backward(self, q, g, v, dy, chunk_states, lengths=None, dstate_out=None, out=None, stream=None):
        """Gradients of the prompt form: (dq, dg, dv, dstate_in), dq None where q is.

        q, g, v, lengths as the prompt had them, chunk_states as it left them;
        dy [B][L][D]: the gradient of y; dstate_out float32 [B][D]: that of the
        state after the prompt, or None.  out: the four tensors to write (None
        for dq without q) instead of new ones; of them dstate_in alone may be an
        input (dstate_out).
        """
        shape, lds = self._inputs(q, g, v, lengths)
        ld_dy = self._rows("dy", dy, shape)
        self._f32("chunk_states", chunk_states, (self.B, -(-shape[1] // hb.HM_RECURRENCE_CHUNK), self.D))
        if dstate_out is not None:
            self._f32("dstate_out", dstate_out, self._state_shape)
        if out is not None:
            if (out[0] is None) != (q is None):
                raise ValueError("dq goes with q")
            self._f32("dstate_in", out[3], self._state_shape)
            ld_out = [0 if t is None else self._rows(name, t, shape) for name, t in zip(("dq", "dg", "dv"), out)]
        else:
            ld_out = (self.D, self.D, self.D)
        return hb._call(self._run_backward, self.device, stream, shape, q, g, v, lds, dy, ld_dy, chunk_states, lengths,
                        dstate_out, out, ld_out)

    def _run_backward(self, shape, q, g, v, lds, dy, ld_dy, chunk_states, lengths, dstate_out, out, ld_out, stream):
        torch, L = self.torch, shape[1]
        if out is None:
            n = 2 if q is None else 3
            grads = torch.empty((n, *shape), dtype=self.tdtype, device=self.device).unbind(0)  # one allocation
            out = (*(() if n == 3 else (None,)), *grads,
                   torch.empty(self._state_shape, dtype=torch.float32, device=self.device))
        dq, dg, dv, dstate_in = out
        with self._ws.order(stream):
            ws, n = self._workspace(L, stream)
            hb._check(self._grads(self._desc_ref, L, None if lengths is None else lengths.data_ptr(),
                                  None if q is None else q.data_ptr(), lds[0], g.data_ptr(), lds[1], v.data_ptr(), lds[2],
                                  dy.data_ptr(), ld_dy, chunk_states.data_ptr(),
                                  None if dstate_out is None else dstate_out.data_ptr(),
                                  None if dq is None else dq.data_ptr(), ld_out[0], dg.data_ptr(), ld_out[1],
                                  dv.data_ptr(), ld_out[2], dstate_in.data_ptr(), None if ws is None else ws.data_ptr(), n,
                                  stream), "hyena_recurrence_backward")
        return out

    def decode_step(self, q, g, v, state, y=None, rows=None, state_out=None, stream=None):
        """One token for every batch row.  Returns y [B][D].

        q (or None), g, v: [B][D] rows with unit element stride.  The state is
        updated in place, or read and written to ``state_out``; with ``rows``
        (int32 [B]) batch row b continues row rows[b] of ``state``, and
        ``state_out`` must be another tensor.
        """
        shape = self._state_shape
        ld_q = 0 if q is None else self._rows("q", q, shape)
        ld_g, ld_v = self._rows("g", g, shape), self._rows("v", v, shape)
        self._f32("state", state, shape)
        if rows is not None:
            hb._expect("rows", rows, self.torch.int32, (self.B,), self.device)
            if state_out is None:
                raise ValueError("rows need a state_out beside the state")
        if state_out is None:
            state_out = state
        else:
            self._f32("state_out", state_out, shape)
        ld_y = self.D if y is None else self._rows("y", y, shape)
        return hb._call(self._run_token, self.device, stream, q, ld_q, g, ld_g, v, ld_v, y, ld_y, state, rows, state_out)

    def _run_token(self, q, ld_q, g, ld_g, v, ld_v, y, ld_y, state, rows, state_out, stream):
        if y is None:
            y = self.torch.empty(self._state_shape, dtype=self.tdtype, device=self.device)
        # (straight to the C entry point: a token's call counts in microseconds)
        hb._check(self._token(self._desc_ref, None if q is None else q.data_ptr(), ld_q, g.data_ptr(), ld_g,
                              v.data_ptr(), ld_v, y.data_ptr(), ld_y, state.data_ptr(),
                              None if rows is None else rows.data_ptr(), state_out.data_ptr(), stream),
                  "hyena_recurrence_decode_step")
        return y
