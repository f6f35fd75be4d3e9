"""Verification of drafted tokens against its definition in float64: whole numbers, compared for equality.

Products u q of two float32 are exact in float64, and so is the sign of u q - p.
Sums of up to 2^17 float64 weights are off by 2^-36 of the whole at most, in any
order: the chance that a number falls that near to a border of the cumulated weights
is below 1e-5 a draw where every token has a border of its own, and the seeds here
are fixed.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import DraftVerify, HMError

pytestmark = pytest.mark.gpu


def verify64(p, tokens, u, q, lengths):
    B, T1, V = p.shape
    T = T1 - 1
    clean = lambda x: np.where(np.isfinite(x) & (x > 0), x, 0.0)  # noqa: E731
    out, counts = np.full((B, T1), -1), np.zeros(B, int)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        k = 0
        while k < n:
            x = tokens[b, k]
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else clean(q[b, k])[x]
            if not u[b, k] * qx < clean(p[b, k])[x]:
                break
            out[b, k] = x
            k += 1
        w = clean(p[b, k])
        if k < n:
            r = np.maximum(w - clean(q[b, k]), 0) if q is not None else w.copy()
            if q is None and 0 <= tokens[b, k] < V:
                r[tokens[b, k]] = 0
            w = r if r.sum() > 0 else w
        sums = np.cumsum(w)
        if sums[-1] > 0:
            over = np.nonzero((sums > u[b, T] * sums[-1]) & (w > 0))[0]
            out[b, k] = over[0] if len(over) else np.nonzero(w > 0)[0][-1]
        counts[b] = k
    return out, counts


def _problem(torch, B, T, V, act, draft_probs=True, seed=0, sharp=3.0):
    g = torch.Generator().manual_seed(B + 10 * T + V + seed)
    x = sharp * torch.randn(B, T + 1, V, generator=g)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    p = torch.softmax(x, -1).to(dt)
    qf = torch.softmax(x[:, :T] + 0.7 * torch.randn(B, T, V, generator=g), -1)
    u = torch.rand(B, T + 1, generator=g)
    if draft_probs:
        tokens = (qf.cumsum(-1) > 0.999 * torch.rand(B, T, 1, generator=g)).int().argmax(-1)
    else:
        tokens = qf.argmax(-1) if T else torch.zeros(B, 0)
    return p, tokens.to(torch.int32), u, qf.to(dt) if draft_probs else None


def _check(torch, p, tokens, u, q, lengths=None, op=None):
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    B, T1, V = p.shape
    op = op or DraftVerify(B, T1 - 1, V)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    got, accepted = op.verify(dev(p), dev(tokens), dev(u), q=dev(q), lengths=dev(n))
    want, counts = verify64(f64(p), tokens.numpy(), f64(u), f64(q), lengths)
    assert (accepted.cpu().numpy() == counts).all(), (accepted.cpu(), counts)
    assert (got.cpu().numpy() == want).all(), (got.cpu(), want)
    return got, accepted


CASES = [(1, 0, 1), (1, 1, 2), (3, 4, 50), (1, 4, 32003), (5, 7, 4096), (7, 3, 4097), (4, 63, 100), (130, 2, 1000),
         (2, 5, 70001), (3, 0, 9999), (2, 1, 131072), (600, 4, 130)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("draft_probs", [True, False])
@pytest.mark.parametrize("B,T,V", CASES)
def test_verify(act, draft_probs, B, T, V):
    torch = require_gpu()
    log(f"verify {act} {draft_probs} {B} {T} {V}")
    p, tokens, u, q = _problem(torch, B, T, V, act, draft_probs)
    _check(torch, p, tokens, u, q)
    g = np.random.default_rng(B + T + V)
    _check(torch, p, tokens, u, q, lengths=list(g.integers(-1, T + 3, B)))


def test_numbers_at_borders():
    """Dyadic probabilities: u q = p refuses, a cumulated weight equal to u of the whole is passed over."""
    torch = require_gpu()
    log("borders")
    p = torch.tensor([[[0.25, 0.25, 0.5, 0.0], [0.0, 0.5, 0.0, 0.5]]]).repeat(7, 1, 1)
    q = torch.tensor([[[0.5, 0.0, 0.25, 0.25]]]).repeat(7, 1, 1)
    tokens = torch.tensor([[0], [0], [0], [2], [3], [1], [2]], dtype=torch.int32)
    u = torch.tensor([[0.5, 0.5], [0.4999, 0.5], [0.5, 0.49999], [0.999, 0.0], [0.0, 0.999], [0.0, 0.25], [0.9, 0.5]])
    got, accepted = _check(torch, p, tokens, u, q)
    assert accepted.tolist() == [0, 1, 0, 1, 0, 1, 1]
    assert got[:, 0].tolist() == [2, 0, 1, 2, 2, 1, 2]
    assert got[1].tolist() == [0, 3] and got[3].tolist() == [2, 1]


def test_weights_that_leave_nothing():
    """p below q all over draws from p; an empty p draws -1; what is no probability counts as 0; tokens that are
    none are refused; numbers outside [0, 1) draw the first or last token that has weight."""
    torch = require_gpu()
    log("nothing left")
    nan, inf = float("nan"), float("inf")
    V = 5000
    p = torch.zeros(8, 2, V)
    q = torch.zeros(8, 1, V)
    tokens = torch.zeros(8, 1, dtype=torch.int32)
    u = torch.full((8, 2), 0.5)
    q[0, 0, :4], p[0, 0, :4] = 0.25, 0.05          # refused, nothing above q
    q[1, 0, 0] = 1.0                               # refused, p is 0
    p[2, 0, 10], p[2, 0, 0], p[2, 0, 4999] = 0.3, nan, inf
    q[2, 0, 0] = 0.7
    p[3, 0, 17], tokens[3, 0] = 1.0, V             # no token
    p[4, 0, 4500], tokens[4, 0], q[4, 0, 3] = 1.0, -1, nan
    p[5, 0, 0], p[5, 1, 4097], p[5, 1, 4999], u[5, 1] = 1.0, 0.5, 0.25, 1.5
    p[6, 0, 0], p[6, 1, 3], p[6, 1, 4999], u[6, 1] = 1.0, 0.5, 0.25, -2.0
    p[7, 0, 0], p[7, 1, 3], p[7, 1, 4200], u[7, 1] = 1.0, 0.5, 0.25, nan
    got, accepted = _check(torch, p, tokens, u, q)
    assert got[:, 0].tolist() == [2, -1, 10, 17, 4500, 0, 0, 0]
    assert got[5:, 1].tolist() == [4999, 3, 4200]
    assert accepted.tolist() == [0, 0, 0, 0, 0, 1, 1, 1]
    _check(torch, p, tokens, u, None)


def test_tokens_are_distributed_as_the_targets():
    """The first token of 40000 verifications of one draft from q: frequencies within 5 standard deviations of p."""
    torch = require_gpu()
    log("distribution")
    B, V = 40000, 12
    g = torch.Generator().manual_seed(11)
    p1, q1 = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(1.5 * torch.randn(V, generator=g), 0)
    tokens = torch.multinomial(q1, B, replacement=True, generator=g).view(B, 1).to(torch.int32)
    u = torch.rand(B, 2, generator=g)
    p, q = p1.expand(B, 2, V).contiguous().cuda(), q1.expand(B, 1, V).contiguous().cuda()
    got, accepted = DraftVerify(B, 1, V).verify(p, tokens.cuda(), u.cuda(), q=q)
    freq = torch.bincount(got[:, 0].cpu(), minlength=V).double() / B
    dev = (p1.double() * (1 - p1.double()) / B).sqrt()
    assert (abs(freq - p1) < 5 * dev).all(), (freq - p1) / dev
    rate = float(torch.minimum(p1, q1).sum())
    assert abs(float(accepted.double().mean()) - rate) < 5 * (rate * (1 - rate) / B) ** 0.5


def test_rows_apart_and_refusals():
    torch = require_gpu()
    log("rows apart")
    p, tokens, u, q = _problem(torch, 3, 4, 333, "f32")
    wide, wq = torch.full((3, 5, 400), 9.0), torch.full((3, 4, 350), 9.0)
    wide[..., 7:340], wq[..., :333] = p, q
    op = DraftVerify(3, 4, 333)
    a = op.verify(p.cuda(), tokens.cuda(), u.cuda(), q=q.cuda())
    out = (torch.empty_like(a[0]), torch.empty_like(a[1]))
    b = op.verify(wide.cuda()[..., 7:340], tokens.cuda(), u.cuda(), q=wq.cuda()[..., :333], out=out)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and b[0] is out[0]
    P, X, N, Q = p.cuda(), tokens.cuda(), u.cuda(), q.cuda()
    for args, kw in (((P[:, :4], X, N), {}), ((P, X.long(), N), {}), ((P, X, N.double()), {}), ((P, X, N[:, :4]), {}),
                     ((P, X, N), dict(q=Q.bfloat16())), ((P.half(), X, N), {}), ((p, X, N), {}),
                     ((P, X, N), dict(lengths=torch.zeros(3, device="cuda"))),
                     ((P[:, :1].expand(3, 5, 333), X, N), {}), ((P.transpose(1, 2).contiguous().transpose(1, 2), X, N), {})):
        with pytest.raises(ValueError):
            op.verify(*args, **kw)
    with pytest.raises(HMError):
        DraftVerify(3, 64, 333)
    with pytest.raises(HMError):
        DraftVerify(3, 4, 0)
    none = DraftVerify(0, 4, 333)
    assert none.verify(P[:0], X[:0], N[:0])[0].shape == (0, 5)


def test_captured_verification_replays():
    torch = require_gpu()
    log("graph")
    op = DraftVerify(6, 4, 9000)
    dev = [t.cuda() for t in _problem(torch, 6, 4, 9000, "f32")]
    call = lambda x: op.verify(x[0], x[1], x[2], q=x[3])  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(dev)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(dev)
    for seed in range(1, 5):
        new = [t.cuda() for t in _problem(torch, 6, 4, 9000, "f32", seed=seed)]
        for a, b in zip(dev, new):
            a.copy_(b)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        call([t.cuda() for t in _problem(torch, 6, 4, 9000, "f32", seed=99)])
        assert all(torch.equal(a, b) for a, b in zip(got, call(new)))
