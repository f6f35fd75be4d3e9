"""Gated recurrence (prompt, token, backward) against the recurrence token by token in float64.

Tolerances, in units u = 2^-24 (half a float32 step).  The factors f and i are off
by at most (|g| + 9) u of themselves: the exponent's argument is rounded once
(|g| u of the exponential), the exponential, the quotient and the sum behind it are
good to two units each, and a square root halves what it is given and adds two.
With M the recurrence over absolute values, a token adds the errors of f and i, two
roundings, and in a scan over chunks a rounding of the product of factors and of
the join: E_t = f_t E_{t-1} + (|g_t| + 14) u M_t bounds every element's error.  The
gradients' recurrences are bounded alike; f' and i' are products and quotients of up
to three such factors, 3 (|g| + 12) u.  A bfloat16 result is rounded once more,
2^-8 of itself.  Beside these bounds, which hold for every element but grow with a
channel's memory, the 2-norm of an error is held to what roundings of random sign
give: some 3000 tokens that count, three roundings each, 100 u = 6e-6, and twice
that where two recurrences follow each other; 2^-8 / sqrt(3) = 2.3e-3 of a
bfloat16 result at most.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import GatedRecurrence, HMError
from distilled_modal_ssm_amd import binding as hb

pytestmark = pytest.mark.gpu

U, T = 2.0 ** -24, 2.0 ** -126
NORM = {"f32": 6e-6, "bf16": 2.4e-3}


def gates(gate, input, g):
    """f, i, df/dg, di/dg in float64."""
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        if gate == "log":
            f, away = np.exp(g), -np.expm1(g)
            df = f
        else:
            f, away = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
            df = f * away
        if input == "free":
            return f, np.ones_like(f), df, np.zeros_like(f)
        if input == "convex":
            return f, away, df, -df
        i = np.sqrt(np.maximum(away * (1 + f), 0))
        return f, i, df, np.where(i > 0, -f * df / np.where(i > 0, i, 1), 0)


def forward64(gate, input, q, g, v, S, n):
    """y, last state, states before each token; and the bounds M and E of h."""
    B, L, D = g.shape
    f, i, _, _ = gates(gate, input, g)
    a = np.minimum(abs(g), 200)
    h, M, E = S.copy(), abs(S), np.zeros_like(S)
    y, before = np.zeros((B, L, D)), np.zeros((B, L, D))
    My, Ey, Mb, Eb = (np.zeros((B, L, D)) for _ in range(4))
    for t in range(L):
        live = (t < n)[:, None]
        before[:, t], Mb[:, t], Eb[:, t] = h, M, E
        new = f[:, t] * h + i[:, t] * v[:, t]
        Mn = f[:, t] * M + i[:, t] * abs(v[:, t])
        En = f[:, t] * E + (a[:, t] + 14) * U * Mn + T * (M + Mn)
        h, M, E = np.where(live, new, h), np.where(live, Mn, M), np.where(live, En, E)
        s = 1 if q is None else q[:, t]
        y[:, t] = np.where(live, s * h, 0)
        My[:, t], Ey[:, t] = np.where(live, abs(s) * M, 0), np.where(live, abs(s) * E, 0)
    return dict(y=y, last=h, Ey=Ey + U * My, Elast=E, before=before, Mb=Mb, Eb=Eb)


def backward64(gate, input, q, g, v, dy, fw, dlast, n):
    B, L, D = g.shape
    f, i, df, di = gates(gate, input, g)
    a = np.minimum(abs(g), 200)
    back, M, E = dlast.copy(), abs(dlast), np.zeros_like(dlast)
    out = {k: np.zeros((B, L, D)) for k in ("dq", "dg", "dv", "Edq", "Edg", "Edv")}
    for t in range(L - 1, -1, -1):
        live = (t < n)[:, None]
        s = 1 if q is None else q[:, t]
        ft, it, vt, dyt = f[:, t], i[:, t], v[:, t], dy[:, t]
        hb_, Mb, Eb = fw["before"][:, t], fw["Mb"][:, t], fw["Eb"][:, t]
        e = (a[:, t] + 14) * U
        fe = e * ft + T
        h, Mh = ft * hb_ + it * vt, ft * Mb + it * abs(vt)
        dh = back + dyt * s
        Md = M + abs(dyt * s)
        Ed = E + 2 * U * Md
        term, Mt = df[:, t] * hb_ + di[:, t] * vt, df[:, t] * Mb + abs(di[:, t] * vt)
        Et = df[:, t] * Eb + 3 * (a[:, t] + 12) * U * Mt + T * (Mb + abs(vt))
        for k, x, ex in (("dq", dyt * h, abs(dyt) * (ft * Eb + e * Mh + U * Mh + T * Mb)),
                         ("dg", dh * term, Ed * Mt + Md * Et + 2 * U * Md * Mt),
                         ("dv", dh * it, Ed * it + e * Md * it)):
            out[k][:, t], out["E" + k][:, t] = np.where(live, x, 0), np.where(live, ex, 0)
        back = np.where(live, ft * dh, back)
        E = np.where(live, ft * Ed + fe * Md, E)
        M = np.where(live, ft * Md, M)
    return dict(out, dstate=back, Edstate=E)


class Problem:
    """Seeded inputs on the device and the float64 answer."""

    def __init__(self, torch, B, L, D, act, gate="sigmoid", input="convex", gated=True, lengths=None, resume=False, pad=0,
                 shift=0, special=None, seed=0, train=False):
        self.op = op = GatedRecurrence(B, D, act, gate=gate, input=input)
        self.act, self.L, self.gate, self.input = act, L, gate, input
        g = torch.Generator().manual_seed(1000 * B + 10 * L + D + seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        ld = 3 * D + pad
        memory = 3 * 1000 ** torch.rand(D, generator=g)
        gates_ = (2 * torch.rand(B, L, D, generator=g) - 1) * 1.0986
        gates_ = torch.log(memory) + gates_ if gate == "sigmoid" else -torch.exp(gates_) / memory
        if special == "reset":
            gates_[:, ::7] = -float("inf")
            gates_[:, 3::11] = -90.0
        if special == "wide":
            gates_ = gates_ * 0 + rn(B, L, D) * 12 if gate == "sigmoid" else -torch.exp(3 * rn(B, L, D))
        if special == "open":
            gates_ = gates_ * 0 + (float("inf") if gate == "sigmoid" else 0.0)
        x = rn(B, L, ld)
        x[..., D:2 * D] = gates_
        buf = torch.zeros(B * L * ld + shift, dtype=op.tdtype)
        buf[shift:] = x.to(op.tdtype).reshape(-1)
        rows = buf.cuda()[shift:].view(B, L, ld)
        self.q, self.g, self.v = (rows[..., k * D:(k + 1) * D] for k in range(3))
        if not gated:
            self.q = None
        self.state = rn(B, D).cuda() if resume else None
        self.dy, self.dlast = rn(B, L, D).to(op.tdtype).cuda(), (rn(B, D).cuda() if resume else None)
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
        n = np.full(B, L) if lengths is None else np.clip(np.array(lengths), 0, L)
        f64 = lambda t: None if t is None else t.detach().cpu().double().numpy()  # noqa: E731
        q, gg, v, dy = (f64(t) for t in (self.q, self.g, self.v, self.dy))
        S = np.zeros((B, D)) if self.state is None else f64(self.state)
        dl = np.zeros((B, D)) if self.dlast is None else f64(self.dlast)
        self.fw = forward64(gate, input, q, gg, v, S, n)
        self.bw = backward64(gate, input, q, gg, v, dy, self.fw, dl, n) if train else None
        if lengths is not None:  # what lies past a row's end does not matter
            for b in range(B):
                for t in (self.q, self.g, self.v, self.dy):
                    if t is not None:
                        t[b, n[b]:] = float("nan")

    def prefill(self, **kw):
        return self.op.prefill(self.q, self.g, self.v, lengths=self.lengths, state_in=self.state, **kw)

    def backward(self, chunks, **kw):
        return self.op.backward(self.q, self.g, self.v, self.dy, chunks, lengths=self.lengths, dstate_out=self.dlast, **kw)

    def compare(self, name, got, ref, bound, act, norms=1):
        got = got.detach().cpu().double().numpy()
        assert np.isfinite(got).all(), name
        if act == "bf16":
            bound = bound + 2.0 ** -8 * (abs(ref) + bound)
        bad = abs(got - ref) - bound
        at = np.unravel_index(bad.argmax(), bad.shape) if bad.size else None
        assert bad.max(initial=0.0) <= 0, f"{name} off by {abs(got - ref)[at]}, bound {bound[at]}, at {at}"
        size = np.linalg.norm(ref)
        if size > 0 and ref.size >= 256:
            err = np.linalg.norm(got - ref) / size
            assert err <= norms * NORM[act], (name, err)

    def check(self, y, last):
        self.compare("y", y, self.fw["y"], self.fw["Ey"], self.act)
        self.compare("state", last, self.fw["last"], self.fw["Elast"], "f32")

    def check_grads(self, dq, dg, dv, dstate):
        if self.q is not None:
            self.compare("dq", dq, self.bw["dq"], self.bw["Edq"], self.act, 2)
        else:
            assert dq is None
        self.compare("dg", dg, self.bw["dg"], self.bw["Edg"], self.act, 2)
        self.compare("dv", dv, self.bw["dv"], self.bw["Edv"], self.act, 2)
        self.compare("dstate", dstate, self.bw["dstate"], self.bw["Edstate"], "f32", 2)


CASES = [
    dict(B=1, L=1, D=1),
    dict(B=3, L=1, D=64, resume=True),
    dict(B=2, L=2, D=33, input="free"),
    dict(B=4, L=5, D=200, lengths=[0, 1, 5, 3], resume=True),
    dict(B=2, L=16, D=130, gate="log", input="norm", resume=True),
    dict(B=2, L=17, D=128, gate="log", input="convex"),
    dict(B=1, L=63, D=96, gated=False),
    dict(B=1, L=64, D=256, input="norm"),
    dict(B=3, L=65, D=70, gate="log", input="free", resume=True, gated=False),
    dict(B=1, L=127, D=128, pad=2),
    dict(B=2, L=128, D=129, pad=1, resume=True),
    dict(B=2, L=129, D=128, shift=1),
    dict(B=1, L=130, D=66, shift=2, pad=2, gate="log", input="norm"),
    dict(B=5, L=300, D=130, lengths=[300, 0, 128, 129, 1], resume=True),
    dict(B=4, L=260, D=64, lengths=[-3, 999, 64, 192], gate="log", input="norm", resume=True),
    dict(B=1, L=4099, D=64, resume=True),
    dict(B=1, L=2500, D=190, gate="log", input="norm", resume=True),
    dict(B=2, L=2000, D=100, input="free", lengths=[2000, 1100], resume=True),
    dict(B=2, L=400, D=128, gate="log", input="norm", special="reset", resume=True),
    dict(B=2, L=400, D=128, gate="log", input="free", special="reset", resume=True, gated=False),
    dict(B=1, L=300, D=128, special="wide", input="norm"),
    dict(B=1, L=300, D=128, gate="log", input="convex", special="wide"),
    dict(B=1, L=200, D=64, special="open", resume=True),
    dict(B=1, L=200, D=64, gate="log", input="norm", special="open", resume=True),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kw", CASES, ids=[",".join(f"{k}={v}" for k, v in c.items()) for c in CASES])
def test_prompt_and_backward(kw, act):
    torch = require_gpu()
    log(f"gated recurrence {act} {kw}")
    p = Problem(torch, act=act, train=True, **kw)
    y, last = p.prefill()
    p.check(y, last)
    chunks = p.op.new_chunk_states(p.L).fill_(float("nan"))
    y2, last2 = p.prefill(chunk_states=chunks)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    p.check_grads(*p.backward(chunks))


@pytest.mark.parametrize("act,lengths", [("f32", None), ("bf16", [20011, 9500])])
def test_long_prompts_and_backward(act, lengths):
    """More than twice 64 places of 128 tokens, and four times backward: several links of the chain between them."""
    torch = require_gpu()
    log(f"long {act}")
    p = Problem(torch, 1 if lengths is None else 2, 20011, 70, act, lengths=lengths, resume=True, train=True)
    chunks = p.op.new_chunk_states(p.L)
    p.check(*p.prefill(chunk_states=chunks))
    p.check_grads(*p.backward(chunks))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("input", ["free", "convex", "norm"])
@pytest.mark.parametrize("B,D,gated,special", [(1, 1, True, None), (3, 300, True, "wide"), (37, 2048, False, None),
                                               (8, 257, True, "reset")])
def test_token(act, gate, input, B, D, gated, special):
    torch = require_gpu()
    log(f"token {act} {gate} {input} {B} {D}")
    p = Problem(torch, B, 1, D, act, gate, input, gated=gated, resume=True, special=special)
    row = lambda t: None if t is None else t[:, 0]  # noqa: E731
    state = p.state.clone()
    y = p.op.decode_step(row(p.q), row(p.g), row(p.v), state)
    p.check(y[:, None], state)
    # beams: each row from another one, and rows out of range from themselves
    rows = torch.arange(B, dtype=torch.int32).flip(0)
    rows[0] = -1
    if B > 1:
        rows[1] = B
    src = torch.where((rows < 0) | (rows >= B), torch.arange(B, dtype=torch.int32), rows)
    out = torch.empty_like(state)
    y2 = p.op.decode_step(row(p.q), row(p.g), row(p.v), p.state, rows=rows.cuda(), state_out=out)
    moved = p.state[src.long().cuda()].contiguous()
    y3 = p.op.decode_step(row(p.q), row(p.g), row(p.v), moved)
    assert torch.equal(y2, y3) and torch.equal(out, moved)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_in_pieces_is_the_prompt(act):
    """A prompt, the same prompt in two calls, and its last tokens one by one; states in place."""
    torch = require_gpu()
    log("pieces")
    p = Problem(torch, 2, 150, 130, act, resume=True)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    state = p.state.clone()
    ys = [p.op.prefill(cut(p.q, a, b), cut(p.g, a, b), cut(p.v, a, b), state_in=state, state_out=state)[0]
          for a, b in ((0, 131), (131, 147))]
    for t in range(147, 150):
        ys.append(p.op.decode_step(p.q[:, t], p.g[:, t], p.v[:, t], state)[:, None])
    p.check(torch.cat(ys, 1), state)


@pytest.mark.parametrize("L", [7, 60, 700])
@pytest.mark.parametrize("D", [2, 3, 127, 129, 131, 255, 257])
def test_odd_numbers_of_channels_and_states_in_place(D, L):
    """Rows that begin between words, two lanes with one channel, states and their gradients replaced."""
    torch = require_gpu()
    log(f"odd {D} {L}")
    p = Problem(torch, 2, L, D, "bf16", lengths=[L, L - 3], resume=True, train=True, shift=1, pad=1)
    chunks = p.op.new_chunk_states(L)
    state = p.state.clone()
    y, last = p.prefill(state_out=state, chunk_states=chunks)
    assert last is state
    p.check(y, last)
    p.state.copy_(state)  # where the prompt left it
    again = p.op.prefill(p.q, p.g, p.v, lengths=p.lengths, state_in=p.state)
    at = p.op.prefill(p.q, p.g, p.v, lengths=p.lengths, state_in=p.state, state_out=p.state)
    assert torch.equal(again[0], at[0]) and torch.equal(again[1], at[1])
    grads = p.backward(chunks)
    p.check_grads(*grads)
    out = (*(torch.empty_like(t) for t in grads[:3]), p.dlast)
    for a, b in zip(p.backward(chunks, out=out), grads):
        assert torch.equal(a, b)


def test_values_that_are_not_finite_stay_in_their_channel():
    torch = require_gpu()
    log("not finite")
    p = Problem(torch, 2, 300, 128, "f32", train=True, resume=True)
    chunks = p.op.new_chunk_states(300)
    clean = (*p.prefill(chunk_states=chunks), *p.backward(chunks))
    p.v[0, 100, 5] = float("nan")
    p.v[1, 299, 9] = float("inf")
    p.g[0, 200, 70] = torch.tensor([-1], dtype=torch.int32).view(torch.float32)[0]  # a NaN of all ones
    y, last = p.prefill(chunk_states=chunks)
    grads = p.backward(chunks)
    for t, c in zip((y, last, *grads), clean):
        same = torch.ones_like(t, dtype=torch.bool)
        for b, ch in ((0, 5), (1, 9), (0, 70)):
            same[b, ..., ch] = False
        assert torch.equal(t[same], c[same])
    assert torch.isnan(y[0, 100:, 5]).all() and torch.equal(y[0, :100, 5], clean[0][0, :100, 5])
    assert torch.isnan(y[0, 200:, 70]).all() and torch.isnan(last[0, 70]) and torch.isinf(last[1, 9])


@pytest.mark.parametrize("L", [5, 1000])
def test_memory_around_the_outputs_stays(L):
    """Outputs as columns of wider rows: what lies beside them is not written."""
    torch = require_gpu()
    log(f"around {L}")
    for act in ("f32", "bf16"):
        p = Problem(torch, 2, L, 67, act, lengths=[L, L // 2], resume=True, train=True)
        new = lambda: torch.full((2, L, 90), 7.0, dtype=p.op.tdtype, device="cuda")  # noqa: E731
        ys, gs = new(), [new() for _ in range(3)]
        chunks = p.op.new_chunk_states(L)
        _, last = p.prefill(y=ys[..., 11:78], chunk_states=chunks)
        p.check(ys[..., 11:78], last)
        out = (*(t[..., 11:78] for t in gs), torch.empty_like(last))
        p.check_grads(*p.backward(chunks, out=out))
        for t in (ys, *gs):
            assert (t[..., :11] == 7).all() and (t[..., 78:] == 7).all()
        # a state past the rows' chunks is left alone too
        kept = torch.full_like(chunks, 3.0)
        p.prefill(chunk_states=kept)
        used = -(-(L // 2) // hb.HM_RECURRENCE_CHUNK)
        assert (kept[1, max(used, 1) + 1:] == 3).all()


def test_empty_and_refused_calls():
    torch = require_gpu()
    op = GatedRecurrence(3, 40, "f32")
    x = torch.randn(3, 0, 40, device="cuda")
    s = torch.randn(3, 40, device="cuda")
    y, last = op.prefill(x, x, x, state_in=s, chunk_states=op.new_chunk_states(0))
    assert y.shape == (3, 0, 40) and torch.equal(last, s)
    grads = op.backward(x, x, x, x, op.new_chunk_states(0), dstate_out=s)
    assert torch.equal(grads[3], s)
    none = GatedRecurrence(0, 40, "f32")
    z = torch.empty(0, 7, 40, device="cuda")
    assert none.prefill(z, z, z)[0].shape == (0, 7, 40)
    x = torch.randn(3, 6, 40, device="cuda")
    with pytest.raises(ValueError):
        op.prefill(x, x, x.bfloat16())
    with pytest.raises(ValueError):
        op.prefill(x, x[:, :5], x)
    with pytest.raises(ValueError):
        op.prefill(x, x, x.transpose(0, 1).contiguous().transpose(0, 1))  # rows of a batch apart
    with pytest.raises(ValueError):
        op.prefill(x, x, x[:, :1].expand(3, 6, 40))
    with pytest.raises(ValueError):
        op.prefill(x, x, x, lengths=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        op.backward(x, x, x, x, op.new_chunk_states(65))
    with pytest.raises(ValueError):
        op.decode_step(x[:, 0], x[:, 0], x[:, 0], s, rows=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(HMError):
        op.decode_step(x[:, 0], x[:, 0], x[:, 0], s, rows=torch.zeros(3, dtype=torch.int32, device="cuda"), state_out=s)
    with pytest.raises(ValueError):
        GatedRecurrence(3, 40, "f16")
    with pytest.raises(ValueError):
        GatedRecurrence(3, 40, "f32", gate="tanh")
    with pytest.raises(HMError):
        GatedRecurrence(3, 0, "f32")


def test_captured_prompts_and_gradients_replay():
    """A prompt with its backward pass in a graph, replayed between eager calls on other inputs."""
    torch = require_gpu()
    log("graph")
    op = GatedRecurrence(2, 200, "f32")
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda: torch.randn(2, 700, 200, generator=gen, device="cuda")  # noqa: E731
    q, g, v, dy = new(), new(), new(), new()
    chunks = op.new_chunk_states(700)

    def step(x):
        y, last = op.prefill(*x[:3], chunk_states=chunks)
        return (y, last, *op.backward(*x, chunks))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step((q, g, v, dy))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step((q, g, v, dy))
    for _ in range(4):
        for t in (q, g, v, dy):
            t.copy_(new())
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        other = step((new(), new(), new(), new()))
        want = step((q, g, v, dy))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert not torch.equal(other[0], want[0])


def test_streams_and_the_same_result_twice():
    torch = require_gpu()
    log("streams")
    p = Problem(torch, 3, 3000, 300, "bf16", resume=True, train=True)
    chunks = p.op.new_chunk_states(p.L)
    want = (*p.prefill(chunk_states=chunks), *p.backward(chunks))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        own = p.op.new_chunk_states(p.L)
        torch.cuda.synchronize()
        got.append((*p.prefill(chunk_states=own, stream=s), *p.backward(own, stream=s)))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
