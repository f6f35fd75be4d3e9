"""The operators of drafted generation from a gated recurrent model, and of its
training: what is measured of them.

Three operators beside the modal Hyena operator, linear attention, the dense
products and beam search:

  recurrence  per batch row and channel, with a state h of one number,
                  h_t = f_t h_{t-1} + i_t v_t,      y_t = q_t h_t
              f = exp(g) or sigmoid(g); i = 1, 1 - f or sqrt(1 - f^2); without
              q, y = h.  Over a prompt or a few drafted tokens ("prompt"), for
              one token, where row b may continue another row's state
              ("token"), and forward and backward ("train");
  dense       a product in 8-bit integers: rows of x and of W (its channels)
              are held as whole multiples of their largest magnitude / 127,
                  y[m][n] = s_m t_n sum_k X[m][k] W[n][k],
              s_m also divided by the row's root mean square where asked;
  verify      drafted tokens x_1 .. x_n of every sequence against the target's
              probabilities p, with given numbers u in [0, 1): x_i is kept while
              u_i q_i(x_i) < p_i(x_i); behind the last one kept comes a token
              drawn from max(p - q, 0) of that place (from p, behind all), the
              first whose cumulated weight exceeds the last u times the whole.

A case is a dict of sizes; `run` takes it through the plain form or, with
``own``, through this repository's entry points.
"""

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------- cases


def _rec(op, batch, channels, act, gate="sigmoid", input="convex", length=1, gated=True, ragged=False, resume=False,
         beams=0):
    c = dict(op=op, batch=batch, channels=channels, act=act, gate=gate, input=input, gated=gated)
    if op == "token":
        c.update(beams=beams)
    else:
        c.update(length=length, ragged=ragged, resume=resume)
    return c


def _dense(rows, outputs, inputs, act, rms=False):
    return dict(op="dense", rows=rows, outputs=outputs, inputs=inputs, act=act, rms=rms)


def _verify(batch, drafts, vocab, act, draft_probs=True, ragged=False):
    return dict(op="verify", batch=batch, drafts=drafts, vocab=vocab, act=act, draft_probs=draft_probs, ragged=ragged)


def listed():
    return [
        # sixty-four users' last tokens and four drafted ones each, some drafts cut short
        dict(_rec("prompt", 64, 2048, "bf16", length=5, ragged=True, resume=True), name="recurrence drafts"),
        # one long document: the prompt itself has to be split to fill the GPU
        dict(_rec("prompt", 1, 4096, "bf16", length=65536), name="recurrence long"),
        # a training step's batch at the width of the 1.3B stack
        dict(_rec("train", 8, 2048, "bf16", length=2048), name="train width 2048"),
        # ragged documents in float32, log decays, states and their gradients carried on
        dict(_rec("train", 6, 1000, "f32", gate="log", input="norm", length=1501, ragged=True, resume=True),
             name="train ragged f32"),
        # one user's next token
        dict(_rec("token", 1, 2048, "bf16"), name="token one"),
        # the batch-256 decode workload's rows, each continuing the state of its beam's parent
        dict(_rec("token", 256, 4096, "bf16", gate="log", input="norm", beams=4), name="token beams"),
        # one user's token and four drafted ones through an in_proj of the 1.3B stack
        dict(_dense(5, 6144, 2048, "bf16", rms=True), name="dense drafts"),
        # sixty-four users' drafts through the vocabulary's head, an odd number of tokens
        dict(_dense(320, 32003, 2048, "bf16"), name="dense head"),
        # sixteen prompts of 2048 tokens through the in_proj
        dict(_dense(32768, 6144, 2048, "bf16", rms=True), name="dense prompt"),
        # a small layer in float32, no size a multiple of anything
        dict(_dense(257, 1001, 515, "f32"), name="dense odd f32"),
        # one user's four drafted tokens
        dict(_verify(1, 4, 32003, "f32"), name="verify one"),
        # a batch of 64 with up to seven drafts over a large vocabulary
        dict(_verify(64, 7, 131072, "f32", ragged=True), name="verify batch"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "train", "token", "dense", "dense", "verify"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "dense":
        inputs, outputs = _spread(rng, 64, 8192), _spread(rng, 64, 32768)
        if rng.random() < 0.5:
            inputs, outputs = -(-inputs // 64) * 64, -(-outputs // 64) * 64
        # at most 2^38 products (the prompt has 1.5 times as many)
        rows = _spread(rng, 1, max(1, min(32768, (1 << 38) // (inputs * outputs))))
        return _dense(rows, outputs, inputs, act, rms=rng.random() < 0.5)
    if op == "verify":
        vocab, drafts = _spread(rng, 1000, 131072), rng.choice([0, 1, 2, 3, 4, 4, 5, 7])
        batch = _spread(rng, 1, max(1, min(256, 64 * 8 * 131072 // ((drafts + 1) * vocab))))
        return _verify(batch, drafts, vocab, act, draft_probs=rng.random() < 0.75, ragged=rng.random() < 0.5)
    kw = dict(act=act, gate=rng.choice(["sigmoid", "log"]), input=rng.choice(["free", "convex", "norm"]),
              gated=rng.random() < 0.75)
    channels = _spread(rng, 16, 4096)
    if rng.random() < 0.6:
        channels = -(-channels // 64) * 64
    if op == "token":
        beams = rng.choice([0, 0, 4, 5])
        batch = _spread(rng, 1, 256)
        return _rec(op, max(1, batch // beams) * beams if beams else batch, channels, beams=beams, **kw)
    # at most 2^25 elements (the long document has 2^28, the width-2048 step 2^25)
    length = _spread(rng, 1, 16384)
    batch = _spread(rng, 1, max(1, min(64, (1 << 25) // (length * channels))))
    if length * channels > 1 << 25:
        length = (1 << 25) // channels
    return _rec(op, batch, channels, length=length, ragged=rng.random() < 0.4, resume=rng.random() < 0.5, **kw)


# ---------------------------------------------------------------- inputs


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _prepare_rec(c, g):
    B, D, dt = c["batch"], c["channels"], DTYPES[c["act"]]
    lead = (B,) if c["op"] == "token" else (B, c["length"])
    # channels remember 3 to 3000 tokens; each token moves that by up to three times either way
    memory = torch.exp(math.log(3) + math.log(1000) * _rand(g, D))
    gate = (2 * _rand(g, *lead, D) - 1) * math.log(3)
    gate = torch.log(memory) + gate if c["gate"] == "sigmoid" else -torch.exp(gate) / memory
    # one projection's output, as a layer has it: [q | g | v] of every token
    x = torch.empty(*lead, 3 * D, dtype=dt, device=DEVICE)
    x[..., :D] = _randn(g, *lead, D)
    x[..., D:2 * D] = gate
    x[..., 2 * D:] = _randn(g, *lead, D)
    s = {"q": x[..., :D] if c["gated"] else None, "g": x[..., D:2 * D], "v": x[..., 2 * D:]}
    s["lengths"] = s["rows"] = s["state"] = s["dstate"] = None
    if c["op"] == "token":
        s["state"] = _randn(g, B, D)
        s["state_out"] = s["state"]
        if c["beams"]:
            n = c["beams"]
            parent = torch.randint(0, n, (B // n, n), generator=g, device=DEVICE)
            s["rows"] = (parent + n * torch.arange(B // n, device=DEVICE)[:, None]).reshape(-1).to(torch.int32)
            s["state_out"] = torch.empty_like(s["state"])
        return s
    if c["ragged"]:
        s["lengths"] = (_rand(g, B) * (c["length"] + 1)).to(torch.int32).clamp_(max=c["length"])
    if c["resume"]:
        s["state"] = _randn(g, B, D)
    if c["op"] == "train":
        s["dy"] = _randn(g, *lead, D, dtype=dt)
        if c["resume"]:
            s["dstate"] = _randn(g, B, D)
    return s


def _quantized64(x):
    """Rows of whole numbers -127 .. 127 (as float64) and the rows' largest magnitudes."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    return torch.round(x * 127.0 / torch.where(amax > 0, amax, 1.0)), amax


def _prepare_dense(c, g):
    dt = DTYPES[c["act"]]
    x = _randn(g, c["rows"], c["inputs"])
    # activations of a trained model: a few channels much larger than the rest, tokens of different sizes
    x *= torch.where(_rand(g, c["inputs"]) < 0.02, 8.0, 1.0) * torch.exp(_randn(g, c["rows"], 1))
    w = (_randn(g, c["outputs"], c["inputs"]) * torch.exp(0.3 * _randn(g, c["outputs"], 1)) / c["inputs"] ** 0.5).to(dt)
    return {"x": x.to(dt), "w": w}


def _prepare_verify(c, g):
    B, T, V, dt = c["batch"], c["drafts"], c["vocab"], DTYPES[c["act"]]
    # a broad body and a few likely tokens a row; the drafting model sees them through some noise
    x = 2.0 * _randn(g, B * (T + 1), V)
    hot = torch.randint(0, V, (B * (T + 1), 24), generator=g, device=DEVICE)
    x.scatter_add_(1, hot, 4.0 + 5.0 * _rand(g, B * (T + 1), 24))
    p = torch.softmax(x, -1).to(dt).view(B, T + 1, V)
    x = x.view(B, T + 1, V)[:, :T]
    x = torch.softmax(x + 0.7 * _randn(g, B, T, V), -1)
    s = {"p": p, "u": _rand(g, B, T + 1), "q": None, "lengths": None}
    # drafts: drawn from the drafting model, or its likeliest tokens
    if c["draft_probs"]:
        at = (x.view(B * T, V).cumsum(-1) > 0.999 * _rand(g, B * T, 1)).int().argmax(-1)
        s["q"] = x.to(dt)
    else:
        at = x.view(B * T, V).argmax(-1) if T else torch.empty(0, device=DEVICE)
    s["drafted"] = at.view(B, T).to(torch.int32)
    if c["ragged"]:
        s["lengths"] = (_rand(g, B) * (T + 1)).to(torch.int32).clamp_(max=T)
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    if c["op"] == "dense":
        s = _prepare_dense(c, g)
    elif c["op"] == "verify":
        s = _prepare_verify(c, g)
    else:
        s = _prepare_rec(c, g)
    s["case"] = c
    # the handle that a program keeps: sizes, scratch memory that later calls use again, weights in 8 bits
    if own:
        if c["op"] == "dense":
            from distilled_modal_ssm_amd.int8 import Int8Dense
            s["handle"] = Int8Dense(s["w"])
        elif c["op"] == "verify":
            from distilled_modal_ssm_amd.drafts import DraftVerify
            s["handle"] = DraftVerify(c["batch"], c["drafts"], c["vocab"], device=DEVICE)
        else:
            from distilled_modal_ssm_amd.recurrence import GatedRecurrence
            s["handle"] = GatedRecurrence(c["batch"], c["channels"], c["act"], gate=c["gate"], input=c["input"],
                                          device=DEVICE)
    elif c["op"] == "dense":
        W, amax = _quantized64(s["w"])
        s["W"], s["w_scale"] = W.to(torch.int8), amax[:, 0].float() / 127.0
    return s


# ---------------------------------------------------------------- plain forms


def _gates(c, g):
    """f, i and their derivatives by g, each without cancellation."""
    if c["gate"] == "log":
        f = g.exp()
        df, away = f, -torch.expm1(g)
        both = -torch.expm1(2 * g)  # 1 - f^2
        dnorm = -f * f / torch.where(both > 0, both, 1.0).sqrt()
    else:
        f, away = torch.sigmoid(g), torch.sigmoid(-g)
        df = f * away
        both = away * (1 + f)
        dnorm = -f * f * (away / (1 + f)).sqrt()
    if c["input"] == "free":
        return f, torch.ones_like(f), df, torch.zeros_like(f)
    if c["input"] == "convex":
        return f, away, df, -df
    return f, both.clamp(min=0).sqrt(), df, torch.where(both > 0, dnorm, 0.0)


def _scan(f, w, h):
    """h_t = f_t h_{t-1} + w_t along dimension 1: chunks side by side, then from chunk to chunk."""
    B, L, D = f.shape
    T = max(1, int(math.sqrt(L)))
    N = -(-L // T)
    if N * T > L:
        f = torch.nn.functional.pad(f, (0, 0, 0, N * T - L), value=1.0)
        w = torch.nn.functional.pad(w, (0, 0, 0, N * T - L))
    f, w = f.reshape(B, N, T, D).clone(), w.reshape(B, N, T, D).clone()
    for t in range(1, T):
        w[:, :, t] += f[:, :, t] * w[:, :, t - 1]
        f[:, :, t] *= f[:, :, t - 1]
    for n in range(N):
        w[:, n] += f[:, n] * h[:, None]
        h = w[:, n, -1]
    return w.reshape(B, N * T, D)[:, :L]


def _plain_rec(s, c):
    """(y, state), and for training the gradients of q (where there is one), g, v and the first state too."""
    B, L, D, dt = c["batch"], c["length"], c["channels"], DTYPES[c["act"]]
    g, v = s["g"].float(), s["v"].float()
    q = s["q"].float() if c["gated"] else None
    f, i, df, di = _gates(c, g)
    w = i * v
    inside = None
    if s["lengths"] is not None:
        inside = (torch.arange(L, device=g.device)[None] < s["lengths"][:, None])[..., None]
        f, w = torch.where(inside, f, 1.0), torch.where(inside, w, 0.0)
    first = s["state"] if s["state"] is not None else torch.zeros(B, D, device=g.device)
    h = _scan(f, w, first)
    y = h if q is None else q * h
    if inside is not None:
        y = y * inside
    y, last = y.to(dt), h[:, -1].contiguous()
    if c["op"] == "prompt":
        return y, last
    dy = s["dy"].float()
    if inside is not None:
        dy = dy * inside
    dlast = s["dstate"] if s["dstate"] is not None else torch.zeros(B, D, device=g.device)
    later = torch.cat([f[:, 1:], torch.ones_like(f[:, :1])], 1)
    dh = _scan(later.flip(1), (dy if q is None else dy * q).flip(1), dlast).flip(1)
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    dg, dv = dh * (df * before + di * v), dh * i
    if inside is not None:
        dg, dv = dg * inside, dv * inside
    grads = dg.to(dt), dv.to(dt), f[:, 0] * dh[:, 0]
    return (y, last, *grads) if q is None else (y, last, (dy * h).to(dt), *grads)


def _plain_token(s, c):
    f, i, _, _ = _gates(c, s["g"].float())
    h = s["state"] if s["rows"] is None else s["state"][s["rows"].long()]
    h = f * h + i * s["v"].float()
    s["state_out"].copy_(h)
    y = h if not c["gated"] else s["q"].float() * h
    return y.to(DTYPES[c["act"]]), s["state_out"]


def _plain_dense(s, c):
    x = s["x"]
    # the borders between whole numbers need 64 bits
    X, amax = _quantized64(x)
    scale = amax.float() / 127.0
    if c["rms"]:
        scale = scale * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS)
    return (torch.matmul(X.float(), s["W"].float().t()) * scale * s["w_scale"]).to(x.dtype)


def _plain_verify(s, c):
    B, T, V = c["batch"], c["drafts"], c["vocab"]
    p, q, u, drafted = s["p"], s["q"], s["u"], s["drafted"].long()
    n = torch.full((B,), T, device=p.device) if s["lengths"] is None else s["lengths"].long()
    row = torch.arange(B, device=p.device)
    px = p[:, :T].gather(2, drafted[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, drafted[..., None])[..., 0].double()
    kept = (u[:, :T].double() * qx < px) & (torch.arange(T, device=p.device)[None] < n[:, None])
    accepted = kept.int().cumprod(-1).sum(-1)
    # the next token, in 64 bits: which token a number falls on is a matter of the last digits
    weight = p[row, accepted].double()
    if T:
        at = accepted.clamp(max=T - 1)
        if q is not None:
            rest = (weight - q[row, at].double()).clamp(min=0)
        else:
            rest = weight.scatter(1, drafted[row, at][:, None], 0.0)
        rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, weight)
        weight = torch.where((accepted < n)[:, None], rest, weight)
    whole = weight.cumsum(-1)
    token = (whole > u[:, T:].double() * whole[:, -1:]).int().argmax(-1)
    place = torch.arange(T + 1, device=p.device)[None]
    tokens = torch.nn.functional.pad(drafted, (0, 1))
    tokens = torch.where(place < accepted[:, None], tokens, torch.where(place == accepted[:, None], token[:, None], -1))
    return tokens.int(), accepted.int()


# ---------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"prompt": _plain_rec, "train": _plain_rec, "token": _plain_token, "dense": _plain_dense,
                "verify": _plain_verify}[c["op"]](s, c)
    handle = s["handle"]
    if c["op"] == "prompt":
        return handle.prefill(s["q"], s["g"], s["v"], lengths=s["lengths"], state_in=s["state"])
    if c["op"] == "train":
        chunks = handle.new_chunk_states(c["length"])
        y, last = handle.prefill(s["q"], s["g"], s["v"], lengths=s["lengths"], state_in=s["state"], chunk_states=chunks)
        grads = handle.backward(s["q"], s["g"], s["v"], s["dy"], chunks, lengths=s["lengths"], dstate_out=s["dstate"])
        return y, last, *(grads if c["gated"] else grads[1:])
    if c["op"] == "token":
        y = handle.decode_step(s["q"], s["g"], s["v"], s["state"], rows=s["rows"],
                               state_out=s["state_out"] if c["beams"] else None)
        return y, s["state_out"]
    if c["op"] == "dense":
        return handle(s["x"], rms_eps=EPS if c["rms"] else None)
    return handle.verify(s["p"], s["drafted"], s["u"], q=s["q"], lengths=s["lengths"])


# ---------------------------------------------------------------- what a pass needs, and its exact answer


def work(case):
    c = case
    e = 2 if c["act"] == "bf16" else 4
    if c["op"] == "dense":
        M, N, K = c["rows"], c["outputs"], c["inputs"]
        return {"bytes": float(e * M * (K + N) + N * K + 4 * N), "flops": 2.0 * M * N * K}
    if c["op"] == "verify":
        B, T, V = c["batch"], c["drafts"], c["vocab"]
        # one row of p a sequence, and one of q where a draft was refused (most of the time)
        rows = B * (1.0 if not c["draft_probs"] or T == 0 else 1.8)
        return {"bytes": rows * V * e + 16.0 * B * (T + 1), "flops": 2.0 * rows * V}
    B, D = c["batch"], c["channels"]
    full = B * D * (1 if c["op"] == "token" else c["length"])
    # ragged rows are half as long on average; what lies past their end is still written (zero)
    read = full * (0.5 if c.get("ragged") else 1.0)
    states = 4.0 * B * D
    n = 3 if c["gated"] else 2
    if c["op"] == "train":
        states *= 1 + 3 * c["resume"]
        return {"bytes": e * (read * (n + 1) + full * (n + 1)) + states, "flops": 30.0 * read}
    if c["op"] == "token":
        # parents that no beam continues are not read
        states *= 2 - ((1 - 1 / c["beams"]) ** c["beams"] if c["beams"] else 0)
    else:
        states *= 1 + c["resume"]
    return {"bytes": e * (read * n + full) + states, "flops": 10.0 * read}


def _exact_rec(s, c):
    """Token after token in 64 bits, and back."""
    B, D = c["batch"], c["channels"]
    token = c["op"] == "token"
    L = 1 if token else c["length"]
    get = lambda x: x.reshape(B, L, D)  # noqa: E731
    log = c["gate"] == "log"

    def at(t):
        """f, i, df/dg, di/dg of position t."""
        g = get(s["g"])[:, t].double()
        f = torch.exp(g) if log else 1 / (1 + torch.exp(-g))
        rest = -torch.expm1(g) if log else 1 / (1 + torch.exp(g))
        df = f if log else f * rest
        if c["input"] == "free":
            return f, torch.ones_like(f), df, torch.zeros_like(f)
        if c["input"] == "convex":
            return f, rest, df, -df
        i = torch.sqrt(rest * (1 + f))
        return f, i, df, torch.where(i > 0, -f * df / i, 0.0)

    h = torch.zeros(B, D, dtype=torch.float64, device=DEVICE)
    if s["state"] is not None:
        h = s["state"].double() if s["rows"] is None else s["state"].double()[s["rows"].long()]
    y = torch.zeros(B, L, D, dtype=torch.float64, device=DEVICE)
    train = c["op"] == "train"
    before = torch.empty(B, L, D, dtype=torch.float64, device=DEVICE) if train else None
    live = None
    if s["lengths"] is not None:
        live = torch.arange(L, device=DEVICE)[None] < s["lengths"][:, None]
    for t in range(L):
        f, i, _, _ = at(t)
        new = torch.addcmul(i * get(s["v"])[:, t].double(), f, h)
        if train:
            before[:, t] = h
        h = new if live is None else torch.where(live[:, t, None], new, h)
        out = h if not c["gated"] else h * get(s["q"])[:, t].double()
        y[:, t] = out if live is None else out * live[:, t, None]
    if token:
        return y[:, 0], h
    if not train:
        return y, h
    dq = torch.zeros_like(y) if c["gated"] else None
    dg, dv = torch.zeros_like(y), torch.zeros_like(y)
    back = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()
    for t in range(L - 1, -1, -1):
        f, i, df, di = at(t)
        v, dy = s["v"][:, t].double(), s["dy"][:, t].double()
        dh = back + (dy * s["q"][:, t].double() if c["gated"] else dy)
        here = torch.ones(B, 1, dtype=torch.bool, device=DEVICE) if live is None else live[:, t, None]
        if c["gated"]:
            dq[:, t] = torch.where(here, dy * (f * before[:, t] + i * v), 0.0)
        dg[:, t] = torch.where(here, dh * (df * before[:, t] + di * v), 0.0)
        dv[:, t] = torch.where(here, dh * i, 0.0)
        back = torch.where(here, f * dh, back)
    return (y, h, dq, dg, dv, back) if c["gated"] else (y, h, dg, dv, back)


def _exact_dense(s, c):
    x, w = s["x"].double(), s["w"].double()
    out = torch.empty(c["rows"], c["outputs"], dtype=torch.float64, device=DEVICE)
    tw = w.abs().max(-1).values
    W = torch.round(w * 127 / torch.where(tw > 0, tw, 1.0)[:, None])
    for m in range(0, c["rows"], 4096):
        part = x[m:m + 4096]
        t = part.abs().max(-1).values / 127
        X = torch.round(part * 127 / torch.where(t > 0, part.abs().max(-1).values, 1.0)[:, None])
        if c["rms"]:
            t = t / torch.sqrt(torch.mean(part * part, -1) + EPS)
        out[m:m + 4096] = t[:, None] * (tw / 127) * torch.mm(X, W.T)
    return out


def _exact_verify(s, c):
    """One sequence and one token after the other."""
    B, T = c["batch"], c["drafts"]
    tokens, counts = torch.full((B, T + 1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    drafted, u = s["drafted"].cpu(), s["u"].double().cpu()
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        k = 0
        while k < n:
            x = int(drafted[b, k])
            q = 1.0 if s["q"] is None else float(s["q"][b, k, x])
            if not float(u[b, k]) * q < float(s["p"][b, k, x]):
                break
            tokens[b, k] = x
            k += 1
        w = s["p"][b, k].double()
        if k < n:
            if s["q"] is not None:
                r = torch.relu(w - s["q"][b, k].double())
            else:
                r = w.clone()
                r[int(drafted[b, k])] = 0
            w = r if bool((r > 0).any()) else w
        sums = torch.cumsum(w, 0)
        tokens[b, k] = int(torch.searchsorted(sums, u[b, T].to(sums.device) * sums[-1], right=True))
        counts[b] = k
    return tokens.to(DEVICE), counts.to(DEVICE)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "dense":
        return _exact_dense(s, c)
    return _exact_verify(s, c) if c["op"] == "verify" else _exact_rec(s, c)
