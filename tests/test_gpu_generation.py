"""More of linear attention and beam search against float64: precision, resets,
graphs, long generation, and the prompt kernel's forms that need larger sizes.

The inputs, the recurrence in float64 and the bounds that every element is held to
are test_gpu_linattn's; what is stricter here is derived at its test.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from test_gpu_linattn import Problem, _prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(B=2, L=200, H=2, dk=128, dv=128, resume=True), dict(B=1, L=77, H=4, dk=64, dv=96, decay="none"),
    dict(B=1, L=150, H=2, dk=256, dv=64, resume=True), dict(B=2, L=130, H=2, dk=32, dv=40, decay="head", pad=3),
    dict(B=1, L=2500, H=2, dk=128, dv=128),
], ids=str)
def test_bf16_y_has_only_its_own_rounding(kw):
    """A bfloat16 y is its terms' float32 sum rounded once: 2^-8 |y| at most.  On the way one
    factor of a term is kept in two bfloat16 parts, each within 2^-8 of what it stands for:
    2^-16 of the term.  So |error| <= 2^-8 |y| + (1 + 2^-8) (2^-16 + float32's bound) M, with M
    the sum of the terms' absolute values."""
    torch = require_gpu()
    p = Problem(torch, act="bf16", **kw)
    log(f"linattn bf16 rounding {kw}")
    y, S = _prefill(p)
    torch.cuda.synchronize()
    p.check(y, S)
    off = abs(y.cpu().double().numpy().reshape(p.y.shape) - p.y)
    most = 2.0 ** -8 * abs(p.y) + (1 + 2.0 ** -8) * (2.0 ** -16 + p.tol) * p.my
    assert (off <= most).all(), float((off - most).max())
