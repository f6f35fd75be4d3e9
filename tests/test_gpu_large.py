"""Tensors of more than 2^31 elements: the same rows in a call of their own, whose offsets are small, give the same
results.  Whole rows and integers are compared for equality; the end of a long prompt begins from the state that
the part before it leaves, whose sums are formed in another order: 100 roundings of float32 (see
test_gpu_recurrence.py) and one step of bfloat16, 2^-7 of a value, where it falls on the other side."""

import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import DraftVerify, GatedRecurrence, Int8Dense

pytestmark = pytest.mark.gpu

PAST = 1 << 31


def _randn(torch, *shape):
    """bfloat16 values made a piece at a time."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for piece in t.view(-1).split(1 << 28):
        piece.normal_()
    return t


def _near(torch, a, b, scale):
    assert float((a.float() - b.float()).abs().max()) <= (2.0 ** -7 + 100 * 2.0 ** -24) * scale


def test_long_prompts_and_their_gradients():
    torch = require_gpu()
    log("large recurrence")
    L, D, cut = 530000, 4096, 520192  # the cut is a whole number of runs
    assert L * D > PAST
    q, g, v, dy = (_randn(torch, 1, L, D) for _ in range(4))
    op = GatedRecurrence(1, D, "bf16")
    chunks = op.new_chunk_states(L)
    y, last = op.prefill(q, g, v, chunk_states=chunks)
    _, state = op.prefill(q[:, :cut], g[:, :cut], v[:, :cut])
    tail = [t[:, cut:].contiguous() for t in (q, g, v, dy)]
    own = op.new_chunk_states(L - cut)
    y2, last2 = op.prefill(*tail[:3], state_in=state, chunk_states=own)
    _near(torch, y[:, cut:], y2, float(y2.abs().max()))
    _near(torch, last, last2, float(last2.abs().max()))
    del y
    grads = op.backward(q, g, v, dy, chunks)
    grads2 = op.backward(*tail, own)
    for a, b in zip(grads[:3], grads2[:3]):
        _near(torch, a[:, cut:], b, float(b.abs().max()))
    head = [t[:, :1024].contiguous() for t in (q, g, v, dy)]
    own = op.new_chunk_states(1024)
    op.prefill(*head[:3], chunk_states=own)
    short = op.backward(*head, own)  # tokens 0 .. 511 hear next to nothing from behind token 1024
    for a, b in zip(grads[:3], short[:3]):
        _near(torch, a[:, :512], b[:, :512], float(b.abs().max()))


def test_many_rows():
    torch = require_gpu()
    log("large batch")
    B, L, D = 260, 2048, 4097
    assert B * L * D > PAST
    q, g, v = (_randn(torch, B, L, D) for _ in range(3))
    y, last = GatedRecurrence(B, D, "bf16").prefill(q, g, v)
    y2, last2 = GatedRecurrence(1, D, "bf16").prefill(q[-1:], g[-1:], v[-1:])
    assert torch.equal(y[-1:], y2) and torch.equal(last[-1:], last2)


def test_products():
    torch = require_gpu()
    log("large products")
    M, K, N = 40000, 60001, 70
    assert M * K > PAST
    x = _randn(torch, M, K)
    op = Int8Dense(_randn(torch, N, K))
    y = op(x, rms_eps=1e-6)
    # (300 rows take the same kernels: the scales' sums are formed alike)
    assert torch.equal(y[-300:], op(x[-300:].contiguous(), rms_eps=1e-6))
    del x, y
    M, K, N = 70000, 100, 32003
    assert M * N > PAST
    x = _randn(torch, M, K)
    op = Int8Dense(_randn(torch, N, K))
    assert torch.equal(op(x)[-300:], op(x[-300:].contiguous()))


def test_verification():
    torch = require_gpu()
    log("large verification")
    B, T, V = 130, 16, 1000003
    assert B * (T + 1) * V > PAST
    p, q = _randn(torch, B, T + 1, V), _randn(torch, B, T, V)  # (below 0 counts as 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(B, T + 1, generator=g, device="cuda") * 0.2
    out, kept = DraftVerify(B, T, V).verify(p, tokens, u, q=q)
    out2, kept2 = DraftVerify(3, T, V).verify(p[-3:], tokens[-3:], u[-3:], q=q[-3:])
    assert torch.equal(out[-3:], out2) and torch.equal(kept[-3:], kept2)
    assert bool((out.gather(1, kept[:, None].long()) >= 0).all())
