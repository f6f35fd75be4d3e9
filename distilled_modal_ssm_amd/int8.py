"""Dense products in 8-bit integers over the C ABI, on torch tensors.

A weight's rows (output channels) are held in 8 bits with a scale each; every
call brings its rows of activations (tokens) to 8 bits the same way, multiplies
in integers and scales the sums.
"""

from __future__ import annotations

import threading
import weakref

from . import binding as hb

# A device's scratch memory, as long as a handle is there.  (A model has two handles a
# layer, and prompts' rows in 8 bits are as large as a layer's weights: one buffer each
# would take what the weights save.)
_shared, _sharing = weakref.WeakValueDictionary(), threading.Lock()


class Int8Dense:
    """y = x W^T of a weight W [outputs][inputs] in 8-bit integers.

    weight: float32 or bfloat16 rows with unit element stride on the GPU, read
    here once, on the given or the current stream, which calls on other streams
    have to wait for.  ``weight8`` (int8, in the library's blocks) and
    ``weight_scale`` [outputs] hold it.
    """

    def __init__(self, weight, stream=None):
        import torch
        self.torch = torch
        if weight.dim() != 2:
            raise ValueError("a weight is [outputs][inputs]")
        self.device = weight.device
        self.N, self.K = int(weight.shape[0]), int(weight.shape[1])
        if self.K < 1 or self.K > hb.HM_INT8_MAX_K:
            raise ValueError(f"1 to {hb.HM_INT8_MAX_K} inputs, got {self.K}")
        self._ws_bytes = {}  # of each number of rows
        self._types = {torch.float32: hb.HM_F32, torch.bfloat16: hb.HM_BF16}
        with _sharing:
            self._ws = _shared.get(self.device)
            if self._ws is None:
                self._ws = _shared[self.device] = hb._Scratch()  # a captured graph has its own
        self._product = hb.load().hyena_dense_int8_rows
        ld, dtype = self._rows("weight", weight, self.N, self.K)
        with hb._On(self.device, stream) as s:
            self.weight8 = torch.empty(hb.hyena_int8_bytes(self.N, self.K), dtype=torch.int8, device=self.device)
            self.weight_scale = torch.empty(self.N, dtype=torch.float32, device=self.device)
            hb.hyena_quantize_rows(self.N, self.K, dtype, weight, ld, 0, 0.0, self.weight8, self.weight_scale, s)

    def _rows(self, name, t, rows, width):
        """Row stride and type of float rows [rows][width]."""
        dtype = self._types.get(t.dtype)
        if dtype is None or t.shape != (rows, width) or t.device != self.device:
            raise ValueError(f"{name}: need float32 or bfloat16 ({rows}, {width}) on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        if t.is_contiguous():
            return width, dtype
        ld = t.stride(0) if rows > 1 else width
        if (width > 1 and t.stride(1) != 1) or ld < width:
            raise ValueError(f"{name}: rows need unit element stride")
        return ld, dtype

    def __call__(self, x, out=None, rms_eps=None, stream=None):
        """y [rows][outputs] of x [rows][inputs], float32 or bfloat16 rows with unit element stride;
        y of x's type, or ``out`` of either, which may share memory with x.

        rms_eps: also scales each row of x by its inverse root mean square, 1 / sqrt(mean x^2 + eps).
        """
        M = int(x.shape[0]) if x.dim() == 2 else -1
        ld, dtype = self._rows("x", x, M, self.K)
        ldo, otype = (self.N, dtype) if out is None else self._rows("out", out, M, self.N)
        return hb._call(self._run, self.device, stream, x, M, ld, dtype, rms_eps, out, ldo, otype)

    def _run(self, x, M, ld, dtype, rms_eps, out, ldo, otype, stream):
        if out is None:
            out = self.torch.empty((M, self.N), dtype=x.dtype, device=self.device)
        n = self._ws_bytes.get(M)
        if n is None:
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            n = self._ws_bytes[M] = hb.hyena_dense_int8_rows_workspace(M, self.K)
        with self._ws.order(stream):
            ws = hb._scratch(self._ws, n, stream, self.device)
            # (straight to the C entry point: a token's call counts in microseconds)
            hb._check(self._product(M, self.N, self.K, dtype, x.data_ptr(), ld, rms_eps is not None, rms_eps or 0.0,
                                    self.weight8.data_ptr(), self.weight_scale.data_ptr(), otype, out.data_ptr(), ldo,
                                    ws.data_ptr(), n, stream), "hyena_dense_int8_rows")
        return out
