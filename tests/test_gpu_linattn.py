"""Linear attention with a decay against the recurrence token by token in float64.

Tolerances.  Every output is a sum of products; M is the same sum over absolute
values (the recurrence on |q|, |k|, |v|, |S_0|), so an error of e in every factor
of every term is at most e M.  float32 operands and the state pass through at
most about dk + 2 * 64 additions and 8 roundings for each 64 tokens of history
that still count (a decay below exp(-17) a chunk leaves nothing of the rest), and
operands kept to 24 bits: (dk + 128 + 8 L / 64 + 16) 2^-24 M.  A bfloat16 y is
rounded once (2^-8 |y|), and its two kinds of terms may each have one factor
rounded to bfloat16 on the way: 2 * 2^-8 M more at most.  Beside these bounds,
which hold for every element, the 2-norm of the error is held to what roundings
of random sign give: 2^-8 / sqrt(3) of a bfloat16 y at most, twice over in
squares (0.0033), and for float32 2^-24 times the square root of the additions
(at most 8 of them in a row of 1024: 4e-6).
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import HMError, LinearAttention
from distilled_modal_ssm_amd import binding as hb

pytestmark = pytest.mark.gpu

NORM = {"f32": 4e-6, "bf16": 3.3e-3}


def _recurrence(q, k, v, a, S, lengths):
    """q [B][L][H][dk], k, v float64; a [B][L][H]; S [B][H][dk][dv] -> y [B][L][H][dv], S."""
    B, L, H, dk = q.shape
    y = np.zeros((B, L, H, v.shape[-1]))
    S = S.copy()
    for b in range(B):
        for t in range(int(lengths[b])):
            S[b] = np.exp(a[b, t])[:, None, None] * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            y[b, t] = np.matmul(q[b, t][:, None, :], S[b])[:, 0]
    return y, S


def _heads64(t, n, H, dim):
    x = t.detach().cpu().double().numpy()
    x = x.reshape(*x.shape[:-1], n, dim)
    return x[..., np.arange(H) * n // H, :]


class Problem:
    """Seeded inputs on the device and the float64 answer."""

    def __init__(self, torch, B, L, H, dk, dv, act, decay="token", qh=None, kh=None, vh=None, resume=False, lengths=None,
                 pad=0, shift=0, special=None, seed=0):
        self.op = LinearAttention(B, H, dk, dv, act, q_heads=qh, k_heads=kh, v_heads=vh)
        op = self.op
        g = torch.Generator().manual_seed(1000 * B + 10 * L + dk + 7 * dv + seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.act, self.L = act, L
        w = (op.q_heads * dk, op.k_heads * dk, op.v_heads * dv)
        # one buffer of fused rows, `pad` spare elements a row, `shift` elements off alignment
        ld = sum(w) + pad
        buf = rn(B * L * ld + shift).to(op.tdtype)
        self.buf = buf.cuda()
        rows = self.buf[shift:].view(B, L, ld)
        self.q, self.k, self.v = rows[..., :w[0]], rows[..., w[0]:w[0] + w[1]], rows[..., w[0] + w[1]:sum(w)]
        if decay == "token":
            a = -torch.exp(rn(B, L, H) * 1.5 - 3.0)
        elif decay == "head":
            a = -torch.exp(rn(H) * 1.5 - 3.0)
        else:
            a = None
        if special == "reset":  # a new document now and then, and one that all but forgets
            a[:, ::7] = -float("inf")
            a[:, 3::11] = -700.0
        if special == "strong":
            a = a * 200.0
        if special == "zero":
            a = a * 0.0
        self.a = None if a is None else a.cuda()
        self.state = rn(B, H, dk, dv).cuda() if resume else None
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
        n = np.full(B, L) if lengths is None else np.clip(np.array(lengths), 0, L)
        if lengths is not None:  # what lies past a row's end does not matter
            for b in range(B):
                for x in (self.q, self.k, self.v):
                    x[b, n[b]:] = float("nan")
                if decay == "token":
                    self.a[b, n[b]:] = float("nan")
        a64 = np.zeros((B, L, H)) if a is None else np.broadcast_to(a.double().numpy(), (B, L, H))
        q64, k64, v64 = (_heads64(x, m, H, d) for x, m, d in ((self.q, op.q_heads, dk), (self.k, op.k_heads, dk),
                                                              (self.v, op.v_heads, dv)))
        S0 = np.zeros((B, H, dk, dv)) if self.state is None else self.state.cpu().double().numpy()
        with np.errstate(invalid="ignore"):
            self.y, self.S = _recurrence(q64, k64, v64, a64, S0, n)
            self.my, self.mS = _recurrence(abs(q64), abs(k64), abs(v64), a64, abs(S0), n)
        self.y, self.my = self.y * op.scale, self.my * abs(op.scale)
        self.tol = (dk + 128 + 8 * L / 64 + 16) * 2.0 ** -24

    def check(self, y, S):
        B, L, H, dv = self.y.shape
        gy = y.detach().cpu().double().numpy().reshape(B, L, H, dv)
        gS = S.detach().cpu().double().numpy()
        ty = self.tol * self.my
        if self.act == "bf16":
            ty = ty + 2.0 ** -8 * (abs(self.y) + 2 * self.my)
        assert np.isfinite(gy).all() and np.isfinite(gS).all()
        bad = abs(gy - self.y) - ty
        assert bad.max(initial=0.0) <= 0, f"y off by {abs(gy - self.y).max()} at {np.unravel_index(bad.argmax(), bad.shape)}"
        bad = abs(gS - self.S) - self.tol * self.mS
        assert bad.max(initial=0.0) <= 0, f"state off by {abs(gS - self.S).max()} at {np.unravel_index(bad.argmax(), bad.shape)}"
        for got, ref, tol in ((gy, self.y, NORM[self.act]), (gS, self.S, NORM["f32"])):
            n = np.linalg.norm(ref)
            if n > 0 and ref.size >= 256:
                assert np.linalg.norm(got - ref) <= tol * n, (np.linalg.norm(got - ref) / n, tol)


def _prefill(p, **kw):
    y, S = p.op.prefill(p.q, p.k, p.v, p.a, lengths=p.lengths, state_in=p.state, **kw)
    return y, S


PROMPTS = [
    dict(B=1, L=1, H=1, dk=1, dv=1),
    dict(B=2, L=1, H=3, dk=16, dv=16, resume=True),
    dict(B=1, L=2, H=4, dk=33, dv=17, decay="head"),
    dict(B=2, L=63, H=2, dk=64, dv=64, decay="none"),
    dict(B=1, L=64, H=2, dk=128, dv=128),
    dict(B=3, L=65, H=2, dk=128, dv=64, resume=True),
    dict(B=1, L=129, H=3, dk=40, dv=24, pad=3),
    dict(B=2, L=200, H=4, dk=100, dv=130, qh=2, kh=1, vh=4, resume=True),
    dict(B=2, L=97, H=2, dk=256, dv=256),
    dict(B=1, L=130, H=2, dk=256, dv=72, decay="head", resume=True),
    dict(B=1, L=70, H=2, dk=8, dv=200, shift=1),
    dict(B=2, L=333, H=8, dk=64, dv=96, qh=8, kh=2, vh=2, lengths=[333, 120]),
    dict(B=5, L=150, H=2, dk=32, dv=48, lengths=[0, 1, 64, 150, 149], resume=True),
    dict(B=4, L=80, H=1, dk=96, dv=80, lengths=[-3, 99, 65, 33], pad=8),
    dict(B=1, L=4099, H=1, dk=64, dv=64),
    dict(B=1, L=2500, H=2, dk=128, dv=128, decay="head", resume=True),
    dict(B=3, L=1800, H=1, dk=128, dv=40, lengths=[1800, 700, 0], resume=True),
    dict(B=1, L=300, H=2, dk=64, dv=64, special="reset", resume=True),
    dict(B=1, L=300, H=2, dk=128, dv=64, special="strong"),
    dict(B=1, L=200, H=2, dk=64, dv=64, special="zero", resume=True),
    dict(B=2, L=77, H=2, dk=64, dv=66, pad=2, shift=2),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kw", PROMPTS, ids=lambda d: "-".join(f"{k}{v}" for k, v in d.items()).replace(" ", ""))
def test_prompt(kw, act):
    torch = require_gpu()
    p = Problem(torch, act=act, **kw)
    log(f"linattn prompt {act} {kw}")
    y, S = _prefill(p)
    torch.cuda.synchronize()
    p.check(y, S)


@pytest.mark.parametrize("L", [100, 3000])
def test_prompt_state_in_place_and_strided_output(L):
    """state_out = state_in, y in a wider buffer at an odd offset: neither may reach its neighbours."""
    torch = require_gpu()
    p = Problem(torch, 2, L, 2, 64, 40, "bf16", resume=True)
    wide = torch.full((2, L, 2 * 40 + 7), 9.0, dtype=torch.bfloat16, device="cuda")
    S = p.state.clone()
    log(f"linattn in place {L}")
    p.op.prefill(p.q, p.k, p.v, p.a, y=wide[..., 3:83], state_in=S, state_out=S)
    torch.cuda.synchronize()
    p.check(wide[..., 3:83], S)
    assert bool((wide[..., :3] == 9).all()) and bool((wide[..., 83:] == 9).all())


def test_prompt_in_pieces_equals_whole():
    """A prompt cut in two, the state carried on, and single tokens after it."""
    torch = require_gpu()
    p = Problem(torch, 2, 150, 4, 64, 64, "f32", kh=2, vh=2)
    op = p.op
    cut = lambda x, i, j: x[:, i:j].contiguous()  # noqa: E731
    log("linattn pieces")
    y1, S = op.prefill(cut(p.q, 0, 70), cut(p.k, 0, 70), cut(p.v, 0, 70), cut(p.a, 0, 70))
    y2, S = op.prefill(cut(p.q, 70, 146), cut(p.k, 70, 146), cut(p.v, 70, 146), cut(p.a, 70, 146), state_in=S)
    ys = [y1, y2]
    for t in range(146, 150):
        ys.append(op.decode_step(p.q[:, t], p.k[:, t], p.v[:, t], S, p.a[:, t].contiguous())[:, None])
    torch.cuda.synchronize()
    p.check(torch.cat(ys, 1), S)


def test_empty_prompt_keeps_the_state():
    torch = require_gpu()
    op = LinearAttention(2, 3, 32, 16, "f32")
    S = torch.randn(2, 3, 32, 16, device="cuda")
    z = lambda n: torch.empty(2, 0, n, device="cuda")  # noqa: E731
    log("linattn empty")
    y, out = op.prefill(z(96), z(96), z(48), state_in=S)
    y0, out0 = op.prefill(z(96), z(96), z(48))
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 48) and torch.equal(out, S) and not bool(out0.any())
    none = LinearAttention(0, 3, 32, 16, "f32")
    y, out = none.prefill(torch.empty(0, 5, 96, device="cuda"), torch.empty(0, 5, 96, device="cuda"),
                          torch.empty(0, 5, 48, device="cuda"))
    assert y.shape == (0, 5, 48) and out.shape == (0, 3, 32, 16)


TOKENS = [
    dict(B=1, H=1, dk=1, dv=1),
    dict(B=3, H=2, dk=33, dv=17),
    dict(B=2, H=4, dk=64, dv=96, decay="head"),
    dict(B=1, H=16, dk=128, dv=128),
    dict(B=5, H=3, dk=40, dv=100, decay="none"),
    dict(B=2, H=4, dk=256, dv=256, qh=1, kh=1),
    dict(B=7, H=4, dk=128, dv=64, qh=4, kh=2, vh=2),
    dict(B=2, H=2, dk=256, dv=36, pad=5, shift=1),
    dict(B=2, H=2, dk=96, dv=200, special="reset"),
    dict(B=70, H=8, dk=64, dv=64),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kw", TOKENS, ids=lambda d: "-".join(f"{k}{v}" for k, v in d.items()))
def test_token(kw, act):
    torch = require_gpu()
    p = Problem(torch, L=1, act=act, resume=True, **kw)
    S = p.state.clone()
    a = p.a if p.a is None or p.a.dim() == 1 else p.a[:, 0]
    log(f"linattn token {act} {kw}")
    y = p.op.decode_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], S, a)
    torch.cuda.synchronize()
    p.check(y[:, None], S)


@pytest.mark.parametrize("dv", [64, 37])
def test_token_continues_parents(dv):
    """Row b reads the state of rows[b]; the source is left as it was; rows out of range count as their own."""
    torch = require_gpu()
    p = Problem(torch, 6, 1, 2, 48, dv, "f32", resume=True)
    rows = torch.tensor([2, 2, 0, 5, -1, 6], dtype=torch.int32, device="cuda")
    src = [2, 2, 0, 5, 4, 5]
    S, out = p.state, torch.empty_like(p.state)
    before = S.clone()
    log("linattn token rows")
    y = p.op.decode_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], S, p.a[:, 0], rows=rows, state_out=out)
    y2 = p.op.decode_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], gathered := S[src].clone(), p.a[:, 0])
    torch.cuda.synchronize()
    assert torch.equal(S, before)
    assert torch.equal(y, y2) and torch.equal(out, gathered)


def test_states_past_2_31_elements():
    """The last batch row of a state of 2.2e9 elements."""
    torch = require_gpu()
    B, H, d = 520, 64, 256
    op = LinearAttention(B, H, d, d, "bf16")
    S = torch.zeros(B, H, d, d, device="cuda")
    S[-1] = torch.randn(H, d, d, generator=torch.Generator().manual_seed(3)).cuda()
    q, k, v = (torch.randn(B, H * d, device="cuda").bfloat16() for _ in range(3))
    one = LinearAttention(1, H, d, d, "bf16")
    S1 = S[-1:].clone()
    log("linattn large state")
    y = op.decode_step(q, k, v, S)
    y1 = one.decode_step(q[-1:], k[-1:], v[-1:], S1)
    torch.cuda.synchronize()
    ref = S1.double() * 0
    ref += k[-1].double().view(H, d, 1) * v[-1].double().view(H, 1, d)
    prev = torch.randn(H, d, d, generator=torch.Generator().manual_seed(3)).cuda().double()
    assert float((S1[0].double() - prev - ref[0]).abs().max()) <= 2.0 ** -20
    assert torch.equal(S[-1:], S1)
    assert float((y[-1:].double() - y1.double()).norm() / y1.double().norm()) <= NORM["bf16"]


def test_rows_past_2_31_elements():
    """A prompt whose rows span 2.4e9 elements, compared with the same rows packed."""
    torch = require_gpu()
    L, ld, d = 60000, 40000, 64
    op = LinearAttention(1, 1, d, d, "bf16")
    buf = torch.empty(L * ld, dtype=torch.bfloat16, device="cuda").view(1, L, ld)
    rows = [buf[..., o:o + d] for o in (0, 20000, 39000)]
    for r in rows:
        r.copy_(torch.randn(1, L, d, device="cuda"))
    a = torch.full((1,), -0.01, device="cuda")
    log("linattn long rows")
    y, S = op.prefill(*rows, a)
    y2, S2 = op.prefill(*[r.contiguous() for r in rows], a)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(S, S2)


def test_same_inputs_same_bits():
    torch = require_gpu()
    p = Problem(torch, 2, 1100, 4, 128, 128, "bf16", resume=True)
    log("linattn determinism")
    one, two = _prefill(p), _prefill(p)
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_other_stream():
    """Calls on a stream of their own, by object and by handle, with torch's allocations made for it."""
    torch = require_gpu()
    p = Problem(torch, 2, 1500, 2, 64, 64, "f32", resume=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    log("linattn stream")
    y, S = _prefill(p, stream=s)
    s.synchronize()
    p.check(y, S)
    y, S = _prefill(p, stream=int(s.cuda_stream))
    s.synchronize()
    p.check(y, S)


def test_graph_replays():
    """A prompt in segments and tokens after it, captured and replayed with eager work between."""
    torch = require_gpu()
    p = Problem(torch, 1, 2500, 2, 128, 128, "bf16", resume=True)
    op = p.op
    y, S = torch.empty(1, 2500, 256, dtype=torch.bfloat16, device="cuda"), op.new_state()
    ts = [torch.empty(1, 256, dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def step():
        op.prefill(p.q, p.k, p.v, p.a, state_in=p.state, y=y, state_out=S)
        for t in range(3):
            op.decode_step(p.q[:, t], p.k[:, t], p.v[:, t], S, p.a[:, t], y=ts[t])

    log("linattn graph eager")
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (y, S, *ts)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    log("linattn graph capture")
    with torch.cuda.graph(graph, stream=side):
        step()
    for r in range(3):
        for x in (y, S, *ts):
            x.fill_(7.0)
        torch.randn(1 << 20, device="cuda").sum().item()
        log(f"linattn graph replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        for x, w in zip((y, S, *ts), want):
            assert torch.equal(x, w)


def test_refusals():
    torch = require_gpu()
    op = LinearAttention(2, 4, 32, 16, "f32")
    q, k, v = (torch.zeros(2, 8, n, device="cuda") for n in (128, 128, 64))
    S = op.new_state()
    a = torch.zeros(4, device="cuda")
    ok = dict(q=q, k=k, v=v)
    for kw in (dict(q=q.bfloat16()), dict(q=q[..., :64]), dict(k=k[:, :7]), dict(v=v.cpu()), dict(log_decay=a.double()),
               dict(log_decay=a[:3]), dict(lengths=torch.zeros(2, device="cuda")), dict(state_in=S[:1]),
               dict(state_in=S.transpose(2, 3).contiguous().transpose(2, 3)), dict(state_out=S.double()),
               dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(q=torch.zeros(2, 128, 8, device="cuda").transpose(1, 2)), dict(y=torch.zeros(2, 8, 63, device="cuda")),
               dict(q=torch.zeros(2, 9, 128, device="cuda")[:, :8])):
        with pytest.raises(ValueError):
            op.prefill(**{**ok, **kw})
    with pytest.raises(ValueError):
        op.decode_step(q[:, 0], k[:, 0], v[:, 0], S, rows=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(HMError) as e:
        op.decode_step(q[:, 0], k[:, 0], v[:, 0], S, rows=torch.zeros(2, dtype=torch.int32, device="cuda"), state_out=S)
    assert e.value.status == hb.HM_ERR_INVALID_ARG
    for bad in (dict(heads=4, q_heads=3), dict(heads=4, key_dim=257)):
        with pytest.raises(HMError):
            LinearAttention(**{**dict(batch=2, heads=4, key_dim=32, value_dim=16, act="f32"), **bad})
    with pytest.raises(ValueError):
        LinearAttention(1, 1, 8, 8, "f16")


SHORT = [
    dict(B=3, L=2, H=2, dk=256, dv=256, resume=True),
    dict(B=2, L=16, H=3, dk=128, dv=96, lengths=[16, 5]),
    dict(B=2, L=17, H=3, dk=128, dv=96, lengths=[17, 5]),
    dict(B=2, L=9, H=2, dk=64, dv=64),
    dict(B=4, L=9, H=2, dk=200, dv=33, pad=1, lengths=[0, 9, 12, -1], resume=True),
    dict(B=70, L=8, H=8, dk=16, dv=16),
    dict(B=80, L=16, H=8, dk=64, dv=128, kh=2, vh=2, qh=8, resume=True),
    dict(B=2, L=15, H=2, dk=256, dv=130, special="reset", resume=True),
    dict(B=1, L=3, H=1, dk=5, dv=3, decay="none"),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kw", SHORT, ids=lambda d: "-".join(f"{k}{v}" for k, v in d.items()).replace(" ", ""))
def test_short_prompt(kw, act):
    """Prompts that the state goes through in registers, and the first that goes in chunks."""
    torch = require_gpu()
    p = Problem(torch, act=act, **kw)
    log(f"linattn short {act} {kw}")
    y, S = _prefill(p)
    torch.cuda.synchronize()
    p.check(y, S)
    if p.state is not None:  # the state in place
        S = p.state.clone()
        y, _ = p.op.prefill(p.q, p.k, p.v, p.a, lengths=p.lengths, state_in=S, state_out=S)
        torch.cuda.synchronize()
        p.check(y, S)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L", [7, 40, 100])
def test_later_tokens_that_would_overflow(act, L):
    """q of the first tokens times k of the later ones passes float32; neither is paired in the sum."""
    torch = require_gpu()
    B, H, dk, dv = 2, 3, 64, 48
    op = LinearAttention(B, H, dk, dv, act)
    g = torch.Generator().manual_seed(L)
    q, k, v = (torch.randn(B, L, H, d, generator=g) for d in (dk, dk, dv))
    first = L // 3
    q[:, :first] *= 1e22
    q[:, first:] *= 1e-22
    k[:, first:] *= 1e22
    q, k, v = (x.reshape(B, L, -1).to(op.tdtype).cuda() for x in (q, k, v))
    a = -torch.rand(B, L, H, generator=g).cuda()
    log(f"linattn later overflow {act} L={L}")
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


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L", [7, 40, 200])
def test_rows_past_the_tokens_are_zero_whatever_the_state(act, L):
    torch = require_gpu()
    B, H, dk, dv = 2, 2, 64, 40
    op = LinearAttention(B, H, dk, dv, act)
    q, k, v = (torch.ones(B, L, H * d, device="cuda", dtype=op.tdtype) for d in (dk, dk, dv))
    state = torch.full((B, H, dk, dv), float("inf"), device="cuda")
    n = torch.tensor([L - 4, 0], dtype=torch.int32, device="cuda")
    log(f"linattn zero rows {act} L={L}")
    y, S = op.prefill(q, k, v, None, lengths=n, state_in=state)
    torch.cuda.synchronize()
    assert not y[0, : L - 4].isfinite().any()
    assert (y[0, L - 4:] == 0).all() and (y[1] == 0).all()
    assert (S == float("inf")).all()
