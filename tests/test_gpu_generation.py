"""More of linear attention and beam search against float64: precision, resets,
graphs, long generation, and the prompt kernel's forms that need larger sizes.

The inputs, the recurrence in float64 and the bounds that every element is held to
are test_gpu_linattn's; what is stricter here is derived at its test.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import binding as hb
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


def _prompt_users(torch):
    """One handle, two problems: calls that write the given outputs, the outputs, and the inputs."""
    ps = [Problem(torch, 1, 2500, 2, 128, 128, "bf16", resume=True, seed=s) for s in (1, 2)]
    op = ps[0].op

    def call(i, out):
        p = ps[i]
        op.prefill(p.q, p.k, p.v, p.a, state_in=p.state, y=out[0], state_out=out[1])

    def longer():
        p = Problem(torch, 1, 4500, 2, 128, 128, "bf16")
        op.prefill(p.q, p.k, p.v, p.a)

    outs = [(torch.empty_like(ps[0].q[..., :256].contiguous()), op.new_state()) for _ in ps]
    return call, longer, outs, [(p.buf, p.a, p.state) for p in ps]


def _select_users(torch):
    from distilled_modal_ssm_amd import BeamSearch
    op = BeamSearch(4, 4, 40009)
    g = torch.Generator().manual_seed(1)
    xs = [(torch.randn(16, 40009, generator=g).cuda(), -torch.rand(4, 4, generator=g).cuda()) for _ in range(2)]

    def call(i, out):
        op.select(*xs[i], out=out)

    outs = [tuple(torch.empty(4, 4, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32, torch.uint8))
            for _ in xs]
    return call, lambda: None, outs, xs


@pytest.mark.parametrize("users", [_prompt_users, _select_users])
def test_graphs_keep_their_scratch(users):
    """Two graphs of one handle, captured on one stream after eager calls there; then a longer eager call, the
    handle dropped, and other tensors in whatever memory is free.  Both replays, on streams of their own at
    once, are right and leave those tensors alone."""
    torch = require_gpu()
    call, longer, outs, inputs = users(torch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    with torch.cuda.stream(side):
        for i, out in enumerate(outs):
            log(f"graph scratch eager {i}")
            call(i, out)
    side.synchronize()
    want = [[x.clone() for x in out] for out in outs]
    for i, out in enumerate(outs):
        log(f"graph scratch capture {i}")
        with torch.cuda.graph(graphs[i], stream=side):
            call(i, out)
    log("graph scratch longer")
    with torch.cuda.stream(side):
        longer()
    side.synchronize()
    del call, longer
    filled = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in [1 << 10, 1 << 16, 1 << 21, 1 << 22] * 8]
    streams = [torch.cuda.Stream() for _ in outs]
    for r in range(4):
        for out in outs:
            for x in out:
                x.fill_(3)
        torch.cuda.synchronize()
        log(f"graph scratch replay {r}")
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            for x, e in zip(out, w):
                assert torch.equal(x, e)
        assert all(bool((x == 77).all()) for x in filled)
    del inputs


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L,reset", [(7, 4), (40, 20), (40, 32), (100, 50), (100, 70), (200, 128), (2500, 1100)])
def test_a_reset_forgets_what_would_overflow(act, L, reset):
    """Keys of 1e22 before a decay of -infinity and queries of 1e22 from it on: q . k and S^T q pass
    float32, but no term of the recurrence pairs them."""
    torch = require_gpu()
    from test_gpu_linattn import _heads64, _recurrence
    from distilled_modal_ssm_amd import LinearAttention
    B, H, dk, dv = 1, 3, 64, 48
    op = LinearAttention(B, H, dk, dv, act)
    g = torch.Generator().manual_seed(L + reset)
    q, k, v = (torch.randn(B, L, H, d, generator=g) for d in (dk, dk, dv))
    k[:, :reset] *= 1e22
    q[:, :reset] *= 1e-22
    q[:, reset:] *= 1e22
    k[:, reset:] *= 1e-22
    q, k, v = (x.reshape(B, L, -1).to(op.tdtype).cuda() for x in (q, k, v))
    a = -torch.rand(B, L, H, generator=g)
    a[:, reset] = -float("inf")
    a = a.cuda()
    log(f"linattn reset overflow {act} L={L} reset={reset}")
    y, S = op.prefill(q, k, v, a)
    torch.cuda.synchronize()
    q64, k64, v64 = (_heads64(x, H, H, d) for x, d in ((q, dk), (k, dk), (v, dv)))
    a64, zero = a.cpu().double().numpy(), np.zeros((B, H, dk, dv))
    ry, rS = _recurrence(q64, k64, v64, a64, zero, [L] * B)
    my, mS = _recurrence(abs(q64), abs(k64), abs(v64), a64, zero, [L] * B)
    ry, my = ry * op.scale, my * op.scale
    tol = (dk + 128 + 8 * L / 64 + 16) * 2.0 ** -24
    ty = tol * my + (2.0 ** -8 * (abs(ry) + 2 * my) if act == "bf16" else 0.0)
    assert (abs(y.cpu().double().numpy().reshape(ry.shape) - ry) <= ty).all()
    assert (abs(S.cpu().double().numpy() - rS) <= tol * mS).all()


# The prompt kernel's forms that smaller problems do not reach: 128 value columns a workgroup over
# several chunks, in one pass and in segments (True), and segments of the narrowest and widest keys.
FORMS = [
    ("bf16", False, dict(B=16, H=16, L=200, dk=128, dv=128)),
    ("bf16", False, dict(B=16, H=16, L=200, dk=100, dv=100, special="reset", resume=True)),  # rows of 8 bytes
    ("bf16", False, dict(B=16, H=16, L=200, dk=100, dv=101, lengths=[200, 0, 64, 65] * 4)),  # of 2
    ("bf16", False, dict(B=8, H=64, L=200, dk=32, dv=128, lengths=[200, 199, 128, 1] * 2, resume=True)),
    ("bf16", True, dict(B=1, H=16, L=1300, dk=128, dv=128, special="reset")),
    ("bf16", True, dict(B=1, H=50, L=800, dk=128, dv=128, special="reset", resume=True)),
    ("bf16", True, dict(B=1, H=50, L=750, dk=100, dv=100, lengths=[733])),
    ("bf16", True, dict(B=1, H=20, L=1300, dk=128, dv=124, kh=4, vh=5, decay="head", resume=True)),
    ("bf16", True, dict(B=2, H=2, L=600, dk=256, dv=72, lengths=[600, 411], resume=True)),
    ("bf16", True, dict(B=2, H=2, L=1500, dk=30, dv=40, special="reset", resume=True)),
    ("bf16", True, dict(B=2, H=2, L=1501, dk=32, dv=130, lengths=[1501, 257], pad=4)),
    ("f32", False, dict(B=6, H=32, L=150, dk=64, dv=128, kh=8, vh=8, lengths=[150, 31, 0, 64, 149, 97], resume=True)),
    ("f32", False, dict(B=6, H=32, L=150, dk=64, dv=70, special="reset")),
    ("f32", False, dict(B=8, H=64, L=100, dk=32, dv=128, decay="none", resume=True)),
    ("f32", True, dict(B=1, H=16, L=700, dk=64, dv=128, special="reset", resume=True)),
    ("f32", True, dict(B=1, H=16, L=700, dk=62, dv=126, lengths=[500])),
    ("f32", True, dict(B=1, H=50, L=450, dk=64, dv=128, lengths=[449], resume=True)),
    ("f32", True, dict(B=1, H=20, L=1000, dk=62, dv=126, special="reset")),
    ("f32", True, dict(B=2, H=2, L=600, dk=256, dv=72, lengths=[600, 411], resume=True)),
    ("f32", True, dict(B=1, H=2, L=900, dk=250, dv=200, special="reset")),
    ("f32", True, dict(B=2, H=4, L=700, dk=30, dv=40, decay="head", lengths=[10, 700])),
]


@pytest.mark.parametrize("act,segments,kw", FORMS, ids=str)
def test_prompt_forms(act, segments, kw):
    torch = require_gpu()
    p = Problem(torch, act=act, **kw)
    assert (hb.hyena_linattn_prefill_workspace(p.op.desc, p.L) > 0) == segments
    log(f"linattn form {act} {kw}")
    y, S = _prefill(p)
    torch.cuda.synchronize()
    p.check(y, S)


def _hybrid(torch, **kw):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from beam_generate import random_model
    return random_model(torch, **kw)


def test_a_search_forms_the_prompts_last_logits_only():
    """No memory for the logits of every position of a long prompt (492 MB here, the rest is below 100)."""
    torch = require_gpu()
    L, V = 30000, 8192
    model = _hybrid(torch, layers=2, width=128, vocab=V, heads=4, modes=8)
    prompt = torch.randint(0, V, (1, L), generator=torch.Generator().manual_seed(1)).cuda()
    model.generate(prompt[:, :100], 2, 2)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    log("hybrid last logits")
    model.generate(prompt, 2, 2)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < L * V * 2 // 2


def test_last_logits_are_the_last_of_all():
    """Both are the same sums in another order, rounded to bfloat16 once: a neighbouring value at most."""
    torch = require_gpu()
    model = _hybrid(torch, layers=2, width=128, vocab=600, heads=4, modes=8)
    prompts = torch.randint(0, 600, (3, 90), generator=torch.Generator().manual_seed(1)).cuda()
    log("hybrid last of all")
    every, states = model.prefill(prompts)
    last, states1 = model.prefill(prompts, last=True)
    torch.cuda.synchronize()
    every = every.view(3, 90, 600)[:, -1]
    assert last.shape == every.shape
    assert bool(((last.float() - every.float()).abs() <= 2.0 ** -7 * every.float().abs() + 2.0 ** -16).all())
    assert all(torch.equal(a, b) for a, b in zip(states, states1))


@pytest.mark.parametrize("piece", [1, 16])
def test_slow_heads_do_not_drift_over_many_tokens(piece):
    """8000 tokens one at a time, and in prompts of 16, through heads that remember 300 to 3000 of them.

    A step rounds the state once, by 2^-24 / sqrt(3) of it at random (2-norm), and the T tokens that a
    head remembers leave sqrt(T / 2) times that: 1.4e-6 for T = 3000, 5e-6 with room for a state that was
    larger before.  A factor that is off by up to 2^-25 the same way at each token leaves T times that."""
    torch = require_gpu()
    from distilled_modal_ssm_amd import LinearAttention
    n, H, d = 8000, 16, 32
    op = LinearAttention(1, H, d, d, "f32")
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(1, n, H * d, generator=g).cuda() for _ in range(3))
    a = -torch.exp(-torch.linspace(5.7, 8.0, H)).cuda()
    S = op.new_state()
    log(f"linattn long generation by {piece}")
    for t in range(0, n, piece):
        if piece == 1:
            op.decode_step(q[:, t], k[:, t], v[:, t], S, a)
        else:
            op.prefill(*(x[:, t:t + piece].contiguous() for x in (q, k, v)), a, state_in=S, state_out=S)
    ref = torch.zeros(H, d, d, dtype=torch.float64, device="cuda")
    f = torch.exp(a.double())[:, None, None]
    for t in range(n):
        ref = f * ref + k[0, t].double().view(H, d, 1) * v[0, t].double().view(H, 1, d)
    off = (S[0].double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert float(off.max()) <= 5e-6, off.tolist()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L", [10, 11, 14, 15])
@pytest.mark.parametrize("kw", [dict(B=40, H=16, dk=256, dv=128, lengths=[15, 3, 14, 0] * 10, resume=True),
                                dict(B=2, H=3, dk=100, dv=33, special="reset", pad=1)], ids=str)
def test_the_longest_short_prompts_and_the_next(act, L, kw):
    torch = require_gpu()
    p = Problem(torch, act=act, L=L, **kw)
    log(f"linattn short or in chunks {act} L={L} {kw}")
    y, S = _prefill(p)
    torch.cuda.synchronize()
    p.check(y, S)


def test_select_with_scores_and_finished_in_place():
    """Eight steps on the same buffers, against the same steps on new ones."""
    torch = require_gpu()
    from distilled_modal_ssm_amd import BeamSearch
    G, K, V = 7, 4, 3001
    op = BeamSearch(G, K, V, end_token=5)
    g = torch.Generator().manual_seed(4)
    scores, finished = op.first_scores(), torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    s, f = scores.clone(), finished.clone()
    tokens, parents = (torch.empty(G, K, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(8):
        x = torch.randn(G * K, V, generator=g).cuda()
        x[:, 5] += 6.0
        log(f"beam in place {step}")
        scores, want_t, want_p, finished = op.select(x, scores, finished)
        op.select(x, s, f, out=(s, tokens, parents, f))
        torch.cuda.synchronize()
        for got, want in ((s, scores), (tokens, want_t), (parents, want_p), (f, finished)):
            assert torch.equal(got, want)
    assert bool(f.any())
