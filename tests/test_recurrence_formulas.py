"""The float64 recurrence that the GPU tests compare with: its gradients against differences."""

import numpy as np
import pytest

from test_gpu_recurrence import backward64, forward64


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("input", ["free", "convex", "norm"])
@pytest.mark.parametrize("gated", [True, False])
def test_gradients_are_the_differences(gate, input, gated):
    rng = np.random.default_rng(4)
    B, L, D = 2, 7, 3
    n = np.array([7, 4])
    x = {k: rng.standard_normal((B, L, D)) for k in "qgv"}
    if gate == "log":
        x["g"] = -np.exp(x["g"])
    S, dy, dl = rng.standard_normal((B, D)), rng.standard_normal((B, L, D)), rng.standard_normal((B, D))

    def loss(x, S):
        r = forward64(gate, input, x["q"] if gated else None, x["g"], x["v"], S, n)
        return (r["y"] * dy).sum() + (r["last"] * dl).sum()

    q = x["q"] if gated else None
    fw = forward64(gate, input, q, x["g"], x["v"], S, n)
    bw = backward64(gate, input, q, x["g"], x["v"], dy, fw, dl, n)
    step = 1e-6
    for k, d in [("q", "dq")] * gated + [("g", "dg"), ("v", "dv"), (None, "dstate")]:
        ref = bw[d]
        base = S if k is None else x[k]
        num = np.zeros_like(base)
        for at in np.ndindex(base.shape):
            moved = [base.copy(), base.copy()]
            moved[0][at] += step
            moved[1][at] -= step
            lo = [loss(x, m) if k is None else loss({**x, k: m}, S) for m in moved]
            num[at] = (lo[0] - lo[1]) / (2 * step)
        # central differences: step^2 times a third derivative of order 10, and 2^-53 * 100 / step
        assert np.allclose(num, ref, rtol=1e-6, atol=1e-7), d
