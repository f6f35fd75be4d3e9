"""Beam search's selection and the reorder of states, against float64 and plain indexing.

Tolerance of a score: s + ((x - max) - log sum).  x - max and the two additions
round once each, the sum of up to 2^18 exponentials (each within 2^-21 of its
value, argument rounding included) is joined in trees and short runs of at most
64 additions, and its logarithm adds one rounding: with m the largest of |s|,
|x - max| and |log sum| this is below 2^-22 m + 2^-17 for every input here.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import BeamSearch, HMError
from distilled_modal_ssm_amd import binding as hb

pytestmark = pytest.mark.gpu

NEVER = float("-inf")


def _scores64(logits, scores, finished, end):
    """[G][K][V] float64 by the definition."""
    G, K = scores.shape
    x = logits.detach().cpu().double().numpy().reshape(G, K, -1)
    x = np.where(np.isnan(x), NEVER, x)
    s = scores.detach().cpu().double().numpy()
    out = np.full(x.shape, NEVER)
    for g in range(G):
        for k in range(K):
            if finished is not None and int(finished[g, k]):
                out[g, k, end] = s[g, k]
                continue
            top = x[g, k].max()
            if s[g, k] == NEVER or top == NEVER:
                continue
            with np.errstate(invalid="ignore"):
                d = np.where(x[g, k] == top, 0.0, x[g, k] - top)
            out[g, k] = s[g, k] + (d - np.log(np.exp(d).sum()))
    return out


def _tol(ref, scores):
    s = scores.detach().cpu().double().numpy()
    m = max(abs(ref[np.isfinite(ref)]).max(initial=0.0), abs(s[np.isfinite(s)]).max(initial=0.0))
    return 2.0 ** -22 * (2 * m + 20) + 2.0 ** -17


def _check(got, logits, scores, finished, end, exact_order=False):
    out_s, tok, par, fin = (x.detach().cpu().numpy() for x in got)
    ref = _scores64(logits, scores, finished, end)
    G, K, V = ref.shape
    n = out_s.shape[1]
    tol = _tol(ref, scores)
    for g in range(G):
        assert tok[g].min() >= 0 and tok[g].max() < V and par[g].min() >= 0 and par[g].max() < K
        flat = par[g].astype(np.int64) * V + tok[g]
        assert len(set(flat.tolist())) == n, "a continuation came twice"
        r = ref[g].reshape(-1)
        mine = r[flat]
        live = np.isfinite(r).sum()
        assert np.isfinite(out_s[g][:min(n, live)]).all() and (out_s[g][live:] == NEVER).all()
        fine = np.isfinite(mine)
        assert np.array_equal(fine, np.isfinite(out_s[g]))
        assert (abs(out_s[g][fine] - mine[fine]) <= tol).all()
        # nothing better was left out, and the order is by score
        rest = np.delete(r, flat)
        if fine.all() and rest.size:
            assert rest.max() <= mine.min() + 2 * tol
        assert (np.diff(out_s[g][fine]) <= 0).all()
        order = np.lexsort((np.arange(r.size), -r))[:n]
        if exact_order:
            assert np.array_equal(flat, order), (flat, order)
        else:  # equal float32 scores: by the lowest index
            same = (np.diff(out_s[g][fine]) == 0)
            assert (np.diff(flat[fine])[same] > 0).all()
        # those of no probability: the lowest ones
        assert np.array_equal(flat[~fine], [i for i in range(r.size) if r[i] == NEVER][:int((~fine).sum())])
        ended = np.zeros(n, bool) if finished is None else finished[g].cpu().numpy().astype(bool)[par[g]]
        assert np.array_equal(fin[g].astype(bool), ended | (tok[g] == end) if end is not None else ended)


CASES = [
    # groups, beams, vocab, select, type, share of beams ended
    (1, 1, 1, 1, "f32", 0.0),
    (1, 1, 7, 7, "bf16", 0.0),
    (3, 2, 5, 4, "f32", 0.5),
    (1, 4, 32003, 4, "bf16", 0.0),
    (2, 5, 10007, 10, "bf16", 0.4),
    (4, 3, 8192, 6, "f32", 0.3),
    (2, 8, 8193, 16, "f32", 0.0),
    (2, 64, 2000, 64, "bf16", 0.2),
    (1, 16, 40001, 64, "f32", 0.0),
    (40, 4, 511, 8, "bf16", 0.3),
    (1, 2, 160000, 3, "bf16", 0.0),
    (30, 8, 70003, 16, "bf16", 0.2),
    (16, 16, 66000, 64, "f32", 0.1),
]


@pytest.mark.parametrize("G,K,V,n,act,share", CASES)
def test_select(G, K, V, n, act, share):
    torch = require_gpu()
    g = torch.Generator().manual_seed(V + 3 * n)
    x = torch.randn(G * K, V, generator=g) * 3
    x[torch.rand(G * K, V, generator=g) < 0.1] = NEVER
    x[:, V // 2] = 1.0
    x = x.to(torch.bfloat16 if act == "bf16" else torch.float32)
    scores = -5 * torch.rand(G, K, generator=g)
    fin = (torch.rand(G, K, generator=g) < share).to(torch.uint8) if share else None
    if fin is not None:
        x.view(G, K, V)[fin.bool()] = float("nan")  # an ended beam's logits are not read
    end = V - 1
    op = BeamSearch(G, K, V, select=n, end_token=end)
    log(f"select {G}x{K}x{V} -> {n} {act}")
    got = op.select(x.cuda(), scores.cuda(), None if fin is None else fin.cuda())
    torch.cuda.synchronize()
    _check(got, x, scores, fin, end)


@pytest.mark.parametrize("act", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "late ties", "constant", "few"])
def test_rows_in_many_batches(kind, act):
    """Rows long and many enough that a workgroup goes through them in batches: better
    and better ones to the end, ties across batches, nearly all taken out."""
    torch = require_gpu()
    G, K, V, n = 32, 8, 70001, 24
    at = torch.arange(V, device="cuda", dtype=torch.float32)
    if kind == "rising":
        x = at / 4096
    elif kind == "falling":
        x = -at / 4096
    elif kind == "late ties":
        x = torch.where(at >= 40000, 3.0, (at % 5) / 8)
    elif kind == "constant":
        x = torch.zeros_like(at)
    else:
        x = torch.full_like(at, NEVER)
        x[[5, 8191, 8192, 8193, 30000, 69999, 70000]] = torch.tensor([1., 2, 2, 2, -4, 0, 3], device="cuda")
    logits = x.to(getattr(torch, act))[None].repeat(G * K, 1)
    scores = (torch.arange(K, device="cuda", dtype=torch.float32) / 64).repeat(G, 1).contiguous()
    log(f"select batches {kind} {act}")
    got = BeamSearch(G, K, V, select=n).select(logits, scores)
    torch.cuda.synchronize()
    for t in got[:3]:  # every group is alike
        assert bool((t == t[:1]).all())
    _check([t[:1] for t in got], logits[:K].cpu(), scores[:1], None, None)
    out, tok, par, _ = (t[0].cpu() for t in got)
    if kind == "constant":  # the best beam's first tokens
        assert par.tolist() == [K - 1] * n and tok.tolist() == list(range(n))
    if kind == "late ties":
        assert par.tolist() == [K - 1] * n and tok.tolist() == list(range(40000, 40000 + n))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ties_go_to_the_lowest_index(dtype):
    """Constant rows (every token ties, more than any list holds), rows of few values, equal beams."""
    torch = require_gpu()
    V = 9001
    x = torch.zeros(4, V)
    x[1] = torch.arange(V) % 3
    x[2, 5000:5100] = 2.0
    x[3] = x[2]
    for n in (1, 4, 64):
        op = BeamSearch(2, 2, V, select=n)
        log(f"select ties {dtype} {n}")
        s = torch.zeros(2, 2)
        got = op.select(x.to(getattr(torch, dtype)).cuda(), s.cuda())
        torch.cuda.synchronize()
        out, tok, par, fin = (t.cpu().numpy() for t in got)
        # beam 1 of the first group: a third of its tokens at the top, above all of beam 0's uniform ones
        assert np.array_equal(tok[0], np.arange(n) * 3 + 2) and (par[0] == 1).all()
        # the second group's beams are equal: the first beam's hundred tokens before the second's
        assert np.array_equal(tok[1], 5000 + np.arange(n)) and (par[1] == 0).all()
        assert not fin.any()
        assert len(set(out[0].tolist())) == 1 and len(set(out[1].tolist())) == 1


def test_masked_rows_infinities_and_nan():
    """Rows that the mask leaves empty or nearly so, the type's lowest value, +infinity, NaN, dead beams."""
    torch = require_gpu()
    V, K, n = 5003, 6, 8
    x = torch.full((K, V), NEVER)
    x[1, 4321] = -7.0                                     # one token left: log probability 0
    x[2, 17] = torch.finfo(torch.float32).min             # one left, at the lowest value
    x[3, 5] = x[3, 9] = float("inf")                      # these two share the row
    x[3, 6] = 3.0
    x[4] = float("nan")                                   # all out
    x[5] = float("nan")
    x[5, 100] = 1.0
    x[5, 200] = 1.0
    scores = torch.tensor([[-1.0, -2.0, -3.0, -4.0, -1.0, NEVER]])
    op = BeamSearch(1, K, V, select=n)
    log("select masks")
    got = op.select(x.cuda(), scores.cuda())
    torch.cuda.synchronize()
    _check(got, x, scores, None, None, exact_order=True)
    out, tok, par, _ = (t.cpu().numpy()[0] for t in got)
    assert (par[0], tok[0]) == (1, 4321) and out[0] == -2.0
    assert list(zip(par[1:4], tok[1:4])) == [(2, 17), (3, 5), (3, 9)]
    assert (out[4:] == NEVER).all() and list(zip(par[4:], tok[4:])) == [(0, 0), (0, 1), (0, 2), (0, 3)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_all_at_the_lowest_value(dtype):
    """A mask of the type's lowest value over a whole row leaves a uniform row, not an empty one."""
    torch = require_gpu()
    dt = getattr(torch, dtype)
    x = torch.full((2, 1000), torch.finfo(dt).min, dtype=dt)
    x[1, 3] = 0.0
    scores = torch.tensor([[0.0, -1.0]])
    log(f"select lowest {dtype}")
    got = BeamSearch(1, 2, 1000, select=4).select(x.cuda(), scores.cuda())
    torch.cuda.synchronize()
    out, tok, par, _ = (t.cpu().numpy()[0] for t in got)
    assert (par[0], tok[0], out[0]) == (1, 3, -1.0)
    assert (par[1:] == 0).all() and tok[1:].tolist() == [0, 1, 2]
    assert abs(out[1:] + np.log(1000.0)).max() <= 2.0 ** -17


def test_first_step_and_all_ended():
    torch = require_gpu()
    G, K, V = 3, 4, 700
    op = BeamSearch(G, K, V, end_token=2)
    x = torch.randn(G * K, V, generator=torch.Generator().manual_seed(5))
    x.view(G, K, V)[:, 1:] = float("nan")  # beams that are not alive are not read
    s = op.first_scores()
    log("select first")
    got = op.select(x.cuda(), s)
    torch.cuda.synchronize()
    _check(got, x, s, None, 2)
    assert not bool(got[2].any())
    fin = torch.ones(G, K, dtype=torch.uint8)
    s = -torch.rand(G, K, generator=torch.Generator().manual_seed(6))
    log("select ended")
    got = op.select(x.cuda(), s.cuda(), fin.cuda())
    torch.cuda.synchronize()
    want = s.sort(dim=1, descending=True)
    assert torch.equal(got[0].cpu(), want.values) and torch.equal(got[2].cpu().long(), want.indices)
    assert bool((got[1] == 2).all()) and bool(got[3].all())


def test_strided_misaligned_logits_and_in_place_scores():
    torch = require_gpu()
    G, K, V = 2, 3, 1001
    for off, dt in ((1, torch.bfloat16), (3, torch.bfloat16), (1, torch.float32)):
        buf = torch.randn(G * K, V + 16, generator=torch.Generator().manual_seed(off)).to(dt)
        buf[:, :off] = 100.0  # neighbours that must not be read as logits
        buf[:, off + V:] = 100.0
        x = buf.cuda()[:, off:off + V]
        scores = torch.tensor([[-1.0, -2.0, -0.5], [0.0, -3.0, -0.25]])
        s = scores.cuda()
        op = BeamSearch(G, K, V)
        out = (s, *(torch.empty(G, K, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.uint8)))
        log(f"select strided {off} {dt}")
        got = op.select(x, s, out=out)
        torch.cuda.synchronize()
        assert got[0] is s
        _check(got, buf[:, off:off + V], scores, None, None)


def test_logits_past_2_31_elements():
    torch = require_gpu()
    K, V, ld = 5, 3001, 600_000_000
    buf = torch.empty((K - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((K, V), (ld, 1))
    x.copy_(torch.randn(K, V, generator=torch.Generator().manual_seed(8)))
    s = torch.zeros(1, K, device="cuda")
    op = BeamSearch(1, K, V, select=9)
    log("select far rows")
    got = op.select(x, s)
    want = op.select(x.contiguous(), s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _check(got, x.contiguous(), s, None, None)


# ------------------------------------------------------------------ reorder


@pytest.mark.parametrize("G,K", [(1, 1), (1, 2), (3, 4), (2, 5), (2, 8), (2, 9), (1, 16), (2, 33), (1, 64)])
def test_reorder(G, K):
    """Buffers of every alignment and of odd sizes, many of them in a call; parents of every kind."""
    torch = require_gpu()
    g = torch.Generator().manual_seed(100 * G + K)
    rows = G * K
    parents = torch.randint(0, K, (G, K), generator=g)
    parents[0] = torch.arange(K).flip(0)  # a permutation without a fixed row
    states = [torch.randn(rows, 4, 8, 16, 2, generator=g), torch.randn(rows, 3000, generator=g),
              torch.randn(rows, 1, generator=g), torch.randint(0, 255, (rows, 333), generator=g, dtype=torch.uint8),
              torch.randn(rows, 7, generator=g).bfloat16(), torch.randn(rows, 0, generator=g),
              torch.randn(rows, 5, generator=g).double()]
    states += [torch.randn(rows, 12 + i, generator=g) for i in range(100)]
    dev = [s.cuda() for s in states]
    shifted = torch.randn(rows * 64 + 1, generator=g)
    dev.append(shifted.cuda()[1:].view(rows, 64))  # 16-byte rows off alignment
    states.append(shifted[1:].view(rows, 64))
    op = BeamSearch(G, K, 10)
    log(f"reorder {G}x{K}")
    op.reorder(parents.int().cuda(), dev)
    torch.cuda.synchronize()
    at = (parents + K * torch.arange(G)[:, None]).reshape(-1)
    for d, s in zip(dev, states):
        assert torch.equal(d.cpu(), s[at])
    assert torch.equal(op.rows(parents.int().cuda()).cpu().long(), at)


def test_reorder_ignores_parents_out_of_range():
    torch = require_gpu()
    s = torch.randn(8, 40, generator=torch.Generator().manual_seed(1))
    parents = torch.tensor([[-1, 0, 4, 7], [3, 2, 2**31 - 1, -2**31]], dtype=torch.int32)
    d = s.cuda()
    log("reorder bounds")
    BeamSearch(2, 4, 10).reorder(parents.cuda(), [d])
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), s[[0, 0, 2, 3, 7, 6, 6, 7]])


def test_reorder_rows_past_2_32_bytes():
    torch = require_gpu()
    d = torch.empty(4, 700_000_000, device="cuda")
    marks = torch.randn(4, 1000, generator=torch.Generator().manual_seed(2))
    d[:, -1000:] = marks.cuda()
    log("reorder large")
    BeamSearch(1, 4, 10).reorder(torch.tensor([[3, 3, 1, 0]], dtype=torch.int32, device="cuda"), [d])
    torch.cuda.synchronize()
    assert torch.equal(d[:, -1000:].cpu(), marks[[3, 3, 1, 0]])


def test_graph_and_stream():
    """A step captured in a graph and replayed with eager work between; the same on a stream of its own."""
    torch = require_gpu()
    G, K, V = 4, 4, 20011
    g = torch.Generator().manual_seed(9)
    x = torch.randn(G * K, V, generator=g).cuda()
    s0 = (-torch.rand(G, K, generator=g)).cuda()
    st0 = torch.randn(G * K, 5000, generator=g).cuda()
    op = BeamSearch(G, K, V, end_token=0)
    out = tuple(torch.empty(G, K, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32, torch.uint8))
    st = st0.clone()

    def step():
        op.select(x, s0, out=out)
        op.reorder(out[2], [st])

    log("beam graph eager")
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, st)]
    side = torch.cuda.Stream()
    st.copy_(st0)
    torch.cuda.synchronize()
    got = op.select(x, s0, stream=side)
    op.reorder(got[2], [st], stream=int(side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, st), want))
    graph = torch.cuda.CUDAGraph()
    log("beam graph capture")
    with torch.cuda.graph(graph, stream=side):
        step()
    for r in range(3):
        for t in out:
            t.zero_()
        st.copy_(st0)
        torch.randn(1 << 20, device="cuda").sum().item()
        log(f"beam graph replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*out, st), want))


def test_refusals():
    torch = require_gpu()
    op = BeamSearch(2, 3, 50, end_token=1)
    x, s = torch.zeros(6, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    f = torch.zeros(2, 3, dtype=torch.uint8, device="cuda")
    for bad in ((x.double(), s, f), (x[:, :49], s, f), (x[:5], s, f), (x.cpu(), s, f), (x, s.double(), f), (x, s[:1], f),
                (x, s, f.int()), (x, s, f.cpu()), (torch.zeros(50, 6, device="cuda").t(), s, f)):
        with pytest.raises(ValueError):
            op.select(*bad)
    with pytest.raises(ValueError):
        op.select(x, s, f, out=(s, s, s, f))
    with pytest.raises(HMError) as e:
        BeamSearch(2, 3, 50).select(x, s, f)  # ended beams without an end token
    assert e.value.status == hb.HM_ERR_INVALID_ARG
    for bad in (dict(beams=65), dict(beams=0), dict(select=65), dict(select=0), dict(vocab=0), dict(groups=-1),
                dict(beams=1, vocab=3, select=4)):
        with pytest.raises(HMError):
            BeamSearch(**{**dict(groups=2, beams=3, vocab=50), **bad})
    par = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for p, st in ((par.long(), [s.view(6, 1)]), (par, [torch.zeros(5, 4, device="cuda")]),
                  (par, [torch.zeros(4, 6, device="cuda").t()]), (par, [torch.zeros(6, 4)])):
        with pytest.raises(ValueError):
            op.reorder(p, st)
