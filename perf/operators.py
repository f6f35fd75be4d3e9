"""The operators of generation with recurrent states: what is measured of them.

Four operators that a program calls beside the modal Hyena operator when it
generates text from layers with a state of constant size:

  prompt   decaying linear attention over a prompt, with the state after it
               S_t = exp(a_t) S_{t-1} + k_t v_t^T,    y_t = scale S_t^T q_t
           for every batch row and head; S [key_dim][value_dim], a_t <= 0 the
           log decay of the head (one a head, or one a token and head);
  token    the same recurrence for one generated token a batch row, where row b
           may continue the state of another row (the parent of a beam);
  select   one step of beam search: the best of beams x vocabulary continuations
           by summed log probability, ties to the lowest (beam, token);
  reorder  the rows of every layer's state permuted by the beams' parents.

A case is a dict of sizes; `run` takes it through the plain form or, with
``own``, through this repository's entry points.
"""

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NEVER = float("-inf")
PLAIN_CHUNK = 128


# ---------------------------------------------------------------- cases


def _attn(op, batch, heads, key_dim, value_dim, act, decay="token", length=1, q_heads=0, k_heads=0, v_heads=0,
          ragged=False, resume=False, beams=0):
    c = dict(op=op, batch=batch, heads=heads, q_heads=q_heads or heads, k_heads=k_heads or heads,
             v_heads=v_heads or heads, key_dim=key_dim, value_dim=value_dim, act=act, decay=decay)
    if op == "prompt":
        c.update(length=length, ragged=ragged, resume=resume)
    else:
        c.update(beams=beams)
    return c


def listed():
    return [
        # one user's short question: latency of a few small launches
        dict(_attn("prompt", 1, 16, 128, 128, "bf16", length=77), name="prompt short"),
        # the width-2048 workload's prompts: a full batch, one workgroup a head and row is enough
        dict(_attn("prompt", 16, 16, 128, 128, "bf16", length=2048), name="prompt width 2048"),
        # one long document: the prompt itself has to be split to fill the GPU
        dict(_attn("prompt", 1, 16, 128, 128, "bf16", length=65536, decay="head"), name="prompt long"),
        # a second turn of ragged chats in float32: keys and values shared by four heads, states carried on
        dict(_attn("prompt", 6, 32, 64, 128, "f32", length=1501, k_heads=8, v_heads=8, ragged=True, resume=True),
             name="prompt ragged f32"),
        # one user's next token
        dict(_attn("token", 1, 16, 128, 128, "bf16"), name="token one"),
        # the batch-256 decode workload
        dict(_attn("token", 256, 16, 128, 128, "bf16"), name="token batch 256"),
        # six groups of eight beams, each continuing its parent's state, queries and keys shared by all heads
        dict(_attn("token", 48, 24, 64, 96, "f32", q_heads=1, k_heads=1, beams=8), name="token beams"),
        # the first step of one user's search: one live beam of four
        dict(op="select", groups=1, beams=4, vocab=32003, select=4, act="bf16", finished=False, first=True,
             name="select first"),
        # a batch of searches in mid-flight, some beams ended
        dict(op="select", groups=16, beams=5, vocab=100003, select=10, act="bf16", finished=True, first=False,
             name="select ended"),
        # a large batch over a large vocabulary, twice as many continuations kept as beams
        dict(op="select", groups=32, beams=8, vocab=131072, select=16, act="f32", finished=False, first=False,
             name="select large"),
        # one user's search over a two-layer model
        dict(op="reorder", groups=1, beams=4, hyena=1, attn=1, channels=2048, heads=16, modes=16, key_dim=128,
             name="reorder one"),
        # a batch of 64 beams over a 24-layer stack, half Hyena, half linear attention
        dict(op="reorder", groups=8, beams=8, hyena=12, attn=12, channels=2048, heads=16, modes=16, key_dim=128,
             name="reorder stack"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "token", "token", "select", "select", "reorder"])
    if op in ("prompt", "token"):
        heads = rng.choice([4, 8, 16, 24, 32])
        shared = rng.choice(["none", "none", "kv", "qk"])
        group = max(1, heads // rng.choice([2, 4, 8]))
        kw = dict(act=rng.choice(["bf16", "bf16", "f32"]), decay=rng.choice(["token", "token", "head", "none"]))
        if shared == "kv":
            kw.update(k_heads=group if heads % group == 0 else 1, v_heads=group if heads % group == 0 else 1)
        elif shared == "qk":
            kw.update(q_heads=1, k_heads=1)
        key_dim = rng.choice([16, 40, 64, 96, 128, 128, 128, 256])
        value_dim = rng.choice([key_dim, key_dim, 64, 128, rng.choice([24, 80, 100, 192])])
        if op == "prompt":
            # at most 2^19 rows of one head (the long document has 2^20)
            length = _spread(rng, 1, 16384)
            batch = _spread(rng, 1, max(1, min(64, (1 << 19) // (length * heads))))
            return _attn(op, batch, heads, key_dim, value_dim, length=length, ragged=rng.random() < 0.4,
                         resume=rng.random() < 0.4, **kw)
        beams = rng.choice([0, 0, 4, 5])
        batch = _spread(rng, 1, 256 * 16 // heads)
        if beams:
            batch = beams * max(1, batch // beams)
        return _attn(op, batch, heads, key_dim, value_dim, beams=beams, **kw)
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        vocab = _spread(rng, 1000, 160000)
        groups = _spread(rng, 1, max(1, min(64, 32 * 8 * 131072 // (beams * vocab))))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, select=beams * rng.choice([1, 1, 2]),
                    act=rng.choice(["bf16", "f32"]), finished=beams > 1 and rng.random() < 0.5, first=False)
    beams = rng.choice([2, 3, 4, 5, 8, 12, 16])
    layers = _spread(rng, 1, 12)
    heads = rng.choice([8, 16])
    return dict(op=op, groups=_spread(rng, 1, max(1, 64 // beams)), beams=beams, hyena=layers,
                attn=rng.choice([0, layers]), channels=heads * rng.choice([64, 128]), heads=heads,
                modes=rng.choice([8, 16]), key_dim=rng.choice([40, 64, 128]))


# ---------------------------------------------------------------- inputs


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE).to(dtype)


def _prepare_attn(c, g):
    B, H, dt = c["batch"], c["heads"], DTYPES[c["act"]]
    dk, dv = c["key_dim"], c["value_dim"]
    lead = (B, c["length"]) if c["op"] == "prompt" else (B,)
    s = {"q": _randn(g, *lead, c["q_heads"] * dk, dtype=dt), "k": _randn(g, *lead, c["k_heads"] * dk, dtype=dt),
         "v": _randn(g, *lead, c["v_heads"] * dv, dtype=dt)}
    # heads forget over 3 to 3000 tokens; a gate of the token moves that by up to three times either way
    rate = torch.exp(torch.empty(H, device=DEVICE).uniform_(math.log(1 / 3000), math.log(1 / 3), generator=g))
    if c["decay"] == "head":
        s["log_decay"] = -rate
    elif c["decay"] == "token":
        gate = torch.empty(*lead, H, device=DEVICE).uniform_(-math.log(3), math.log(3), generator=g)
        s["log_decay"] = -rate * gate.exp()
    else:
        s["log_decay"] = None
    s["lengths"] = s["rows"] = s["state"] = None
    if c["op"] == "prompt":
        if c["ragged"]:
            u = torch.empty(B, device=DEVICE).uniform_(0.0, 1.0, generator=g)
            s["lengths"] = (u * (c["length"] + 1)).to(torch.int32).clamp_(max=c["length"])
        if c["resume"]:
            s["state"] = _randn(g, B, H, dk, dv)
        s["y"] = torch.empty(B, c["length"], H * dv, dtype=dt, device=DEVICE)
        s["state_out"] = torch.empty(B, H, dk, dv, device=DEVICE)
    else:
        s["state"] = _randn(g, B, H, dk, dv)
        s["y"] = torch.empty(B, H * dv, dtype=dt, device=DEVICE)
        if c["beams"]:
            n = c["beams"]
            parent = torch.randint(0, n, (B // n, n), generator=g, device=DEVICE)
            s["rows"] = (parent + n * torch.arange(B // n, device=DEVICE)[:, None]).reshape(-1).to(torch.int32)
            s["state_out"] = torch.empty_like(s["state"])
        else:
            s["state_out"] = s["state"]
    return s


def _scores64(c, logits, scores, finished):
    """Every continuation's score in 64 bits, [groups][beams][vocab]."""
    G, K, V = c["groups"], c["beams"], c["vocab"]
    x = logits.view(G, K, V).double()
    s = scores.double()[:, :, None] + torch.log_softmax(x, -1)
    if finished is not None:
        ended = finished.bool()[:, :, None]
        at_end = (torch.arange(V, device=x.device) == c["vocab"] - 1)[None, None]
        s = torch.where(ended, torch.where(at_end, scores.double()[:, :, None], NEVER), s)
    return s


def _apart(c, logits, scores, finished, g):
    """Moves beams' scores a little until no two beams' best continuations are
    within 1e-4 of each other: which of two such comes first would be a matter
    of rounding, in any form."""
    G, K, n = c["groups"], c["beams"], c["select"]
    for _ in range(20):
        best = []
        for i in range(G):  # a group at a time: 64-bit scores of all groups are large
            sl = slice(i * K, (i + 1) * K)
            one = dict(c, groups=1)
            s = _scores64(one, logits[sl], scores[i:i + 1], None if finished is None else finished[i:i + 1])[0]
            best.append(s.topk(min(n + 1, c["vocab"]), dim=-1).values)
        best = torch.stack(best)
        beam = torch.arange(K, device=DEVICE)[None, :, None].expand_as(best).reshape(G, -1)
        v, at = best.reshape(G, -1).sort(dim=-1, descending=True)
        beam = beam.gather(1, at)
        m = min(n + 1, v.shape[1])
        near = (v[:, :m - 1] - v[:, 1:m] < 1e-4) & (beam[:, :m - 1] != beam[:, 1:m])
        near = near & torch.isfinite(v[:, 1:m])
        if not bool(near.any()):
            break
        move = torch.empty(G, K, device=DEVICE).uniform_(-0.05, 0.05, generator=g)
        scores = torch.where(near.any(-1)[:, None], scores + move, scores)
    return scores


def _prepare_select(c, g):
    G, K, V, dt = c["groups"], c["beams"], c["vocab"], DTYPES[c["act"]]
    # a broad body and a few likely tokens a row, as a language model's head gives; float32 ones come in steps of 2^-10
    x = 2.0 * torch.randn(G * K, V, generator=g, device=DEVICE)
    hot = torch.randint(0, V, (G * K, 24), generator=g, device=DEVICE)
    x.scatter_add_(1, hot, 4.0 + 5.0 * torch.rand(G * K, 24, generator=g, device=DEVICE))
    x = (x * 1024).round_().div_(1024)
    # tokens that a grammar or a filter has taken out, of every row
    x.masked_fill_(torch.rand(V, generator=g, device=DEVICE)[None] < 0.02, NEVER)
    x[:, V - 1] = 1.0
    logits = x.to(dt)
    scores = -3.0 - 4.0 * torch.rand(G, K, generator=g, device=DEVICE)
    finished = None
    if c["first"]:
        scores = torch.full((G, K), NEVER, device=DEVICE)
        scores[:, 0] = 0.0
    if c["finished"]:
        finished = (torch.rand(G, K, generator=g, device=DEVICE) < 0.25).to(torch.uint8)
        finished[:, 0] = 0
    scores = _apart(c, logits, scores, finished, g)
    return {"logits": logits, "scores": scores, "finished": finished}


def _prepare_reorder(c, g):
    rows, P = c["groups"] * c["beams"], c["channels"] // c["heads"]
    s = {"parents": torch.randint(0, c["beams"], (c["groups"], c["beams"]), generator=g, device=DEVICE).to(torch.int32)}
    s["states"] = [_randn(g, rows, c["heads"], c["modes"], P, 2) for _ in range(c["hyena"])]
    s["states"] += [_randn(g, rows, c["heads"], c["key_dim"], P) for _ in range(c["attn"])]
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    if c["op"] in ("prompt", "token"):
        s = _prepare_attn(c, g)
    elif c["op"] == "select":
        s = _prepare_select(c, g)
    else:
        s = _prepare_reorder(c, g)
    s["case"] = c
    if own:  # the handle that a program keeps: sizes, and scratch memory that later calls use again
        if c["op"] in ("prompt", "token"):
            from distilled_modal_ssm_amd.linear_attention import LinearAttention
            s["handle"] = LinearAttention(c["batch"], c["heads"], c["key_dim"], c["value_dim"], c["act"],
                                          q_heads=c["q_heads"], k_heads=c["k_heads"], v_heads=c["v_heads"],
                                          device=DEVICE)
        else:
            from distilled_modal_ssm_amd.beam import BeamSearch
            sel = c["op"] == "select"
            s["handle"] = BeamSearch(c["groups"], c["beams"], c["vocab"] if sel else 1,
                                     select=c["select"] if sel else 1, end_token=c["vocab"] - 1 if sel else 0,
                                     device=DEVICE)
    return s


# ---------------------------------------------------------------- plain forms


def _heads(x, n, H, dim):
    """[..., n * dim] of n heads as float32 [..., H, dim]: head h takes head h n / H."""
    x = x.float().unflatten(-1, (n, dim))
    return x.repeat_interleave(H // n, dim=-2) if n != H else x


def _decay_between(a):
    """exp of the sums of a [..., T] over j < i <= t, for every j <= t: [..., t, j]; 0 for j > t.
    Each sum starts at j, so a long history costs it no digits."""
    T = a.shape[-1]
    later = torch.ones(T, T, dtype=torch.bool, device=a.device).tril(-1)
    sums = a[..., :, None].expand(*a.shape, T).masked_fill(~later, 0.0).cumsum(-2)
    return sums.masked_fill(~torch.ones(T, T, dtype=torch.bool, device=a.device).tril(), NEVER).exp()


def _plain_prompt(s, c):
    B, L, H, dk, dv = c["batch"], c["length"], c["heads"], c["key_dim"], c["value_dim"]
    q = _heads(s["q"], c["q_heads"], H, dk)
    k = _heads(s["k"], c["k_heads"], H, dk)
    v = _heads(s["v"], c["v_heads"], H, dv)
    a = s["log_decay"]
    a = torch.zeros(B, L, H, device=q.device) if a is None else a.expand(B, L, H)
    inside = None
    if s["lengths"] is not None:
        inside = torch.arange(L, device=q.device)[None, :] < s["lengths"][:, None]
        k, a = k * inside[:, :, None, None], a * inside[:, :, None]
    T = min(PLAIN_CHUNK, L)
    N = -(-L // T)
    pad = N * T - L
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).unflatten(1, (N, T)).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = cut(q), cut(k), cut(v)  # [B][H][N][T][dim]
    a = cut(a[..., None])[..., 0]
    D = _decay_between(a)
    y = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * D, v)
    own_state = torch.matmul((k * D[..., -1, :, None]).transpose(-1, -2), v)  # each chunk's own, at its end
    first = torch.zeros(B, H, 1, dk, dv, device=q.device) if s["state"] is None else s["state"][:, :, None]
    whole = torch.nn.functional.pad(a.sum(-1), (1, 0))  # [B][H][1 + N]; the first state decays by nothing
    every = torch.cat([first, own_state], 2).flatten(-2)
    every = torch.matmul(_decay_between(whole), every).unflatten(-1, (dk, dv))  # the states at all chunk bounds
    y = y + torch.matmul(q, every[:, :, :-1]) * a.cumsum(-1).exp()[..., None]
    y = y * dk ** -0.5
    y = y.permute(0, 2, 3, 1, 4).reshape(B, N * T, H * dv)[:, :L]
    if inside is not None:
        y = y * inside[:, :, None]
    return y.to(s["q"].dtype), every[:, :, -1].contiguous()


def _plain_token(s, c):
    B, H, dk, dv = c["batch"], c["heads"], c["key_dim"], c["value_dim"]
    q = _heads(s["q"], c["q_heads"], H, dk)
    k = _heads(s["k"], c["k_heads"], H, dk)
    v = _heads(s["v"], c["v_heads"], H, dv)
    S = s["state"] if s["rows"] is None else s["state"][s["rows"].long()]
    if s["log_decay"] is not None:
        S = S * s["log_decay"].exp().expand(B, H)[:, :, None, None]
    S = S + k[..., :, None] * v[..., None, :]
    y = (q[..., :, None] * S).sum(-2) * dk ** -0.5
    s["state_out"].copy_(S)
    return y.to(s["q"].dtype).reshape(B, H * dv), s["state_out"]


def _plain_select(s, c):
    G, K, V, n = c["groups"], c["beams"], c["vocab"], c["select"]
    x = s["logits"].float().view(G, K, V)
    x = x - x.amax(-1, keepdim=True)
    score = s["scores"][:, :, None] + (x - x.exp().sum(-1, keepdim=True).log())
    token = torch.arange(V, device=x.device)
    ended = torch.zeros(G, K, dtype=torch.bool, device=x.device)
    if s["finished"] is not None:
        ended = s["finished"].bool()
        kept = torch.where(token == V - 1, s["scores"][:, :, None], NEVER)
        score = torch.where(ended[:, :, None], kept, score)
    # one whole number that orders by score, then by the lowest (beam, token)
    bits = (score + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits) * 4294967296
    order = order.view(G, K * V) - torch.arange(K * V, device=x.device)
    at = order.topk(n, dim=-1).indices
    parents, tokens = at // V, at % V
    ended = ended.gather(1, parents) | (tokens == V - 1)
    return score.view(G, K * V).gather(1, at), tokens.int(), parents.int(), ended.to(torch.uint8)


def _plain_reorder(s, c):
    rows = (s["parents"].long() + c["beams"] * torch.arange(c["groups"], device=s["parents"].device)[:, None]).view(-1)
    return [x.copy_(x[rows]) for x in s["states"]]


# ---------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"prompt": _plain_prompt, "token": _plain_token, "select": _plain_select,
                "reorder": _plain_reorder}[c["op"]](s, c)
    if c["op"] == "prompt":
        return s["handle"].prefill(s["q"], s["k"], s["v"], s["log_decay"], lengths=s["lengths"], y=s["y"],
                                   state_in=s["state"], state_out=s["state_out"])
    if c["op"] == "token":
        if s["rows"] is None:
            y = s["handle"].decode_step(s["q"], s["k"], s["v"], s["state"], s["log_decay"], y=s["y"])
        else:
            y = s["handle"].decode_step(s["q"], s["k"], s["v"], s["state"], s["log_decay"], y=s["y"], rows=s["rows"],
                                        state_out=s["state_out"])
        return y, s["state_out"]
    if c["op"] == "select":
        return s["handle"].select(s["logits"], s["scores"], s["finished"])
    s["handle"].reorder(s["parents"], s["states"])
    return s["states"]


# ---------------------------------------------------------------- what a pass needs, and its exact answer


def work(case):
    c = case
    if c["op"] in ("prompt", "token"):
        e = 2 if c["act"] == "bf16" else 4
        B, H, dk, dv = c["batch"], c["heads"], c["key_dim"], c["value_dim"]
        # ragged prompts are half as long on average; rows past their end are still written (zero)
        tokens = B * (c["length"] * (0.5 if c["ragged"] else 1.0) if c["op"] == "prompt" else 1)
        moved = tokens * e * ((c["q_heads"] + c["k_heads"]) * dk + c["v_heads"] * dv)
        moved += e * H * dv * B * (c["length"] if c["op"] == "prompt" else 1)
        moved += 4 * H * (tokens if c["decay"] == "token" else 1 if c["decay"] == "head" else 0)
        states = (1 + c["resume"]) * B if c["op"] == "prompt" else 2 * B
        if c["op"] == "token" and c["beams"]:  # parents that no beam continues are not read
            states = B * (2 - (1 - 1 / c["beams"]) ** c["beams"])
        return {"bytes": moved + 4.0 * states * H * dk * dv, "flops": 4.0 * tokens * H * dk * dv}
    if c["op"] == "select":
        live = c["groups"] * c["beams"] * (0.8 if c["finished"] else 1.0)
        return {"bytes": live * c["vocab"] * (2.0 if c["act"] == "bf16" else 4.0), "flops": 3.0 * live * c["vocab"]}
    K = c["beams"]
    row = 8 * c["channels"] * c["modes"] * c["hyena"] + 4 * c["channels"] * c["key_dim"] * c["attn"]
    # beams that stay in place are neither read nor written; a parent of several is read once
    return {"bytes": float(c["groups"] * row * ((K - 1) + K * (1 - (1 - 1 / K) ** (K - 1)))), "flops": 0.0}


def _exact_recurrence(s, c):
    """Token after token in 64 bits."""
    B, H, dk, dv = c["batch"], c["heads"], c["key_dim"], c["value_dim"]
    prompt = c["op"] == "prompt"
    L = c["length"] if prompt else 1
    pick = lambda n: torch.arange(H, device=DEVICE) * n // H  # noqa: E731
    get = lambda x, n, d: x.reshape(B, L, n, d)[:, :, pick(n)]  # noqa: E731
    q, k, v = get(s["q"], c["q_heads"], dk), get(s["k"], c["k_heads"], dk), get(s["v"], c["v_heads"], dv)
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEVICE)
    if s["state"] is not None:
        S = s["state"].double() if s["rows"] is None else s["state"].double()[s["rows"].long()]
    a = s["log_decay"]
    a = torch.zeros(1, 1, H, device=DEVICE) if a is None else a
    a = a.reshape(-1, L, H) if c["decay"] == "token" else a.reshape(1, 1, H).expand(1, L, H)
    y = torch.zeros(B, L, H, dv, dtype=torch.float64, device=DEVICE)
    for t in range(L):
        new = torch.exp(a[:, t].double())[..., None, None] * S
        new.addcmul_(k[:, t].double()[..., None], v[:, t].double()[..., None, :])
        out = torch.matmul(q[:, t].double()[..., None, :], new)[..., 0, :]
        if s["lengths"] is not None:
            live = (s["lengths"] > t)[:, None, None]
            out, new = out * live, torch.where(live[..., None], new, S)
        y[:, t], S = out, new
    y = y.reshape(B, L, H * dv) / math.sqrt(dk)
    return (y if prompt else y[:, 0]), S


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] in ("prompt", "token"):
        return _exact_recurrence(s, c)
    if c["op"] == "select":
        kept = []
        for i in range(c["groups"]):
            sl = slice(i * c["beams"], (i + 1) * c["beams"])
            f = None if s["finished"] is None else s["finished"][i:i + 1]
            all_ = _scores64(dict(c, groups=1), s["logits"][sl], s["scores"][i:i + 1], f).flatten()
            kept.append(all_.topk(c["select"]).values)
        return torch.stack(kept), None, None, None
    out = []
    for x in s["states"]:
        rows = [int(p) + i * c["beams"] for i, line in enumerate(s["parents"].tolist()) for p in line]
        out.append(torch.stack([x[r] for r in rows]).double())
    return out
