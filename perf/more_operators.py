"""Measured cases of the delta-rule language-model operators.

Beside the selective scan stands the other recurrence of today's recurrent
language models, the gated delta rule, whose outputs are normed and gated head
by head; and beside the scores of given tokens stands what decides them when
several continuations of a prompt are followed at once: the selection over beams
and vocabulary, and the reordering of every layer's state by its result.  Every
case is one call of one of these operators, on the tensors a program has in hand
at that point.

With ``own`` false the operators run in their plain form (elementary torch
operations in 32 bits, in 64 where 32 lose what matters, rounded once at the
end); with ``own`` true through the entry points of ``recurrent_nn_amd``.
``exact`` is the definition in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64              # steps that the plain form of the delta rule takes together
KEY_EPS = 1e-6          # under the root of a key's norm
NORM_EPS = 1e-6
EOS = 2


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A long prompt of one request through a delta-rule layer: queries and
        # keys as the convolution gives them, gates as the projection does.
        {"name": "delta_prompt", "op": "delta", "batch": 1, "steps": 8192, "key_heads": 16, "heads": 32,
         "dk": 128, "dv": 128, "raw": True, "state": False, "ragged": False, "dtype": "bf16"},
        # Chunks of unlike lengths that go on from earlier states, in 32 bits,
        # keys of norm 1 and decays in hand, as an evaluation runs it.
        {"name": "delta_ragged", "op": "delta", "batch": 8, "steps": 1000, "key_heads": 8, "heads": 8,
         "dk": 64, "dv": 64, "raw": False, "state": True, "ragged": True, "dtype": "f32"},
        # Two odd-sized continuations.
        {"name": "delta_odd", "op": "delta", "batch": 2, "steps": 777, "key_heads": 3, "heads": 6,
         "dk": 96, "dv": 100, "raw": True, "state": True, "ragged": False, "dtype": "f16"},
        # One new token for each of 64 running requests: reading and writing the states.
        {"name": "delta_step", "op": "delta", "batch": 64, "steps": 1, "key_heads": 16, "heads": 32,
         "dk": 128, "dv": 128, "raw": True, "state": True, "ragged": False, "dtype": "bf16"},
        # The layer's outputs, normed head by head and gated.
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "groups": 32, "dim": 128, "gate": "after",
         "shared": True, "dtype": "bf16"},
        # A few tokens of a selective-state layer, gated and then normed as one odd group.
        {"name": "norm_odd", "op": "norm", "rows": 64, "groups": 1, "dim": 5001, "gate": "before",
         "shared": True, "dtype": "f16"},
        # A step of beam search for 32 requests.
        {"name": "beam_batch", "op": "beam", "batch": 32, "beams": 8, "keep": 8, "vocab": 131072,
         "finished": False, "masked": False, "fresh": False, "dtype": "bf16"},
        # One request, twice as many continuations as beams, some of them
        # finished, part of the vocabulary masked out by a grammar.
        {"name": "beam_one", "op": "beam", "batch": 1, "beams": 4, "keep": 8, "vocab": 100001,
         "finished": True, "masked": True, "fresh": False, "dtype": "f32"},
        # The states of a model after that step: windows and delta states of
        # eight layers for 8 requests of 4 beams.
        {"name": "reorder_model", "op": "reorder", "kind": "delta", "batch": 8, "beams": 4, "keep": 4,
         "layers": 8, "dim": 8192, "heads": 32, "dk": 128, "dtype": "bf16"},
        # The hidden and cell states of two bidirectional layers, rows in the middle.
        {"name": "reorder_lstm", "op": "reorder", "kind": "lstm", "batch": 4, "beams": 4, "keep": 4,
         "layers": 2, "dim": 1024, "heads": 0, "dk": 0, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "norm", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "delta":
        dk = rng.choice([128, 128, 64, 96, 32, 256, rng.randint(8, 256)])
        dv = rng.choice([128, 128, 64, 256, rng.randint(8, 256)])
        key_heads = _log(rng, 1, 32)
        heads = key_heads * rng.choice([1, 1, 2, 3])
        batch = _log(rng, 1, 64)
        steps = 1 if rng.random() < 0.3 else _log(rng, 2, 8192)
        most = min(8192 * 32 * 128 * 128 // (dk * dv), 8192 * 32)
        steps = max(1, min(steps, most // (batch * heads)))
        return {"op": op, "batch": batch, "steps": steps, "key_heads": key_heads, "heads": heads,
                "dk": dk, "dv": dv, "raw": rng.random() < 0.6, "state": steps == 1 or rng.random() < 0.5,
                "ragged": batch > 1 and steps > 1 and rng.random() < 0.5, "dtype": dtype}
    if op == "norm":
        dim = rng.choice([64, 128, 256, _log(rng, 16, 8192), _log(rng, 16, 8192)])
        groups = 1 if dim > 512 else _log(rng, 1, 64)
        rows = max(1, min(_log(rng, 1, 16384), 8192 * 4096 // (groups * dim)))
        return {"op": op, "rows": rows, "groups": groups, "dim": dim,
                "gate": rng.choice(["after", "after", "before", "none"]), "shared": rng.random() < 0.6,
                "dtype": dtype}
    if op == "beam":
        vocab = _log(rng, 1000, 262144)
        beams = rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
        batch = max(1, min(_log(rng, 1, 128), 32 * 8 * 131072 // (beams * vocab)))
        return {"op": op, "batch": batch, "beams": beams, "keep": min(64, beams * rng.choice([1, 1, 2])),
                "vocab": vocab, "finished": rng.random() < 0.4, "masked": rng.random() < 0.4,
                "fresh": rng.random() < 0.2, "dtype": dtype}
    kind = rng.choice(["delta", "lstm", "expand"])
    beams = 1 if kind == "expand" else rng.choice([2, 3, 4, 5, 8])
    keep = rng.choice([2, 4, 8]) if kind == "expand" else beams
    batch, layers = _log(rng, 1, 32), rng.randint(1, 12)
    dim = _log(rng, 64, 8192)
    heads, dk = (0, 0) if kind == "lstm" else (_log(rng, 1, 32), rng.choice([32, 64, 100, 128]))
    each = 4 * batch * max(beams, keep) * (heads * dk * dk + 8 * dim)
    layers = max(1, min(layers, (1 << 29) // each))
    return {"op": op, "kind": kind, "batch": batch, "beams": beams, "keep": keep, "layers": layers,
            "dim": dim, "heads": heads, "dk": dk, "dtype": dtype}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE, dtype=torch.float32)

    def whole(hi, *shape):
        return torch.randint(0, hi, shape, generator=gen, device=DEVICE, dtype=torch.int32)

    s = {"case": case}
    if case["op"] == "delta":
        b, t, g, h, dk, dv = (case[k] for k in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
        # rows of the convolution's outputs: queries, keys and values side by side
        rows = torch.nn.functional.silu(normal(b, t, 2 * g * dk + h * dv, dtype=torch.float32))
        q, k, v = rows.split([g * dk, g * dk, h * dv], 2)
        q, k = q.unflatten(2, (g, dk)), k.unflatten(2, (g, dk))
        v = v.unflatten(2, (h, dv))
        size = torch.exp(uniform(h) * math.log(100.0) + math.log(1e-3))     # step sizes 0.001 to 0.1
        A, bias = -(1 + 15 * uniform(h)), size + torch.log(-torch.expm1(-size))
        if case["raw"]:
            rows = rows.to(dt)
            q, k, v = rows.split([g * dk, g * dk, h * dv], 2)
            s["q"], s["k"], s["v"] = q.unflatten(2, (g, dk)), k.unflatten(2, (g, dk)), v.unflatten(2, (h, dv))
            gates = normal(b, t, 2 * h)             # rows of the projection that gives both
            s["g"], s["beta"], s["A"], s["dt_bias"] = gates[:, :, :h], gates[:, :, h:], A, bias
        else:
            for name, x in (("q", q), ("k", k)):
                s[name] = (x / x.norm(dim=3, keepdim=True).clamp(min=1e-6)).to(dt)
            s["v"] = v.to(dt).contiguous()
            s["g"] = A * torch.nn.functional.softplus(normal(b, t, h, dtype=torch.float32) + bias)
            s["beta"] = torch.sigmoid(normal(b, t, h, dtype=torch.float32))
            s["A"] = s["dt_bias"] = None
        s["state"] = normal(b, h, dk, dv, dtype=torch.float32) * 0.3 if case["state"] else None
        s["lens"] = None
        if case["ragged"]:
            # at least one full row, and one of no steps where there are three rows or more
            s["lens"] = whole(t, b) + 1
            s["lens"][0] = t
            if b > 2:
                s["lens"][-1] = 0
    elif case["op"] == "norm":
        r, g, n = case["rows"], case["groups"], case["dim"]
        s["x"] = (normal(r, g, n, dtype=torch.float32) * torch.exp(0.5 * normal(n, dtype=torch.float32))).to(dt)
        s["weight"] = 0.5 + (uniform(n) if case["shared"] else uniform(g, n))
        # rows of the projection that gives the gate behind other columns
        s["z"] = None if case["gate"] == "none" else normal(r, g * n + 64)[:, 64:].unflatten(1, (g, n))
    elif case["op"] == "beam":
        b, n, v = case["batch"], case["beams"], case["vocab"]
        logits = 2.5 * normal(b, n, v, dtype=torch.float32)
        if case["masked"]:
            logits.masked_fill_(uniform(b, n, v) < 0.5, -math.inf)
        s["logits"] = logits.to(dt)
        s["scores"] = -(20 * uniform(b, 1) + 2 * uniform(b, n))     # sums of earlier tokens' log probabilities
        if case["fresh"]:                           # the first step: all beams are the same prompt
            s["scores"][:, 1:] = -math.inf
        s["finished"] = uniform(b, n) < 0.3 if case["finished"] else None
    else:
        b, n, k, d = case["batch"], case["beams"], case["keep"], case["dim"]
        rows, s["states"] = b * n, []
        s["dim"] = 1 if case["kind"] == "lstm" else 0
        for _ in range(case["layers"]):
            if case["kind"] == "lstm":              # [directions, rows, hidden]
                s["states"] += [normal(2, rows, d), normal(2, rows, d)]
            else:
                s["states"] += [normal(rows, 3, d),
                                normal(rows, case["heads"], case["dk"], case["dk"], dtype=torch.float32)]
        # many beams stay where they are
        stay = torch.arange(k, device=DEVICE, dtype=torch.int32).clamp(max=n - 1).expand(b, k)
        s["parents"] = torch.where(uniform(b, k) < 0.4, stay, whole(n, b, k))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"delta": _plain_delta, "norm": _plain_norm, "beam": _plain_beam,
            "reorder": _plain_reorder}[c["op"]](c, state)


def _own(c, s):
    import recurrent_nn_amd as ra
    if c["op"] == "delta":
        o, h = ra.gated_delta(s["q"], s["k"], s["v"], s["beta"], g=s["g"], A=s["A"], dt_bias=s["dt_bias"],
                              beta_sigmoid=c["raw"], normalize=c["raw"], state=s["state"],
                              sequence_lens=s["lens"])
        return {"o": o, "state": h}
    if c["op"] == "norm":
        return {"y": ra.gated_norm(s["x"], s["weight"], z=s["z"], gate_first=c["gate"] == "before",
                                   eps=NORM_EPS)}
    if c["op"] == "beam":
        got = ra.beam_select(s["logits"], s["scores"], keep=c["keep"], finished=s["finished"], eos=EOS)
        return {"scores": got.scores, "tokens": got.tokens, "parents": got.parents}
    return {"states": ra.reorder_states(s["states"], s["parents"], dim=s["dim"])}


def _plain_delta(c, s):
    b, t, h, dv = c["batch"], c["steps"], c["heads"], c["dv"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    beta, g = s["beta"].float(), s["g"].float()
    if c["raw"]:
        q = q * torch.rsqrt((q * q).sum(3, keepdim=True) + KEY_EPS)
        k = k * torch.rsqrt((k * k).sum(3, keepdim=True) + KEY_EPS)
        beta = 1 / (1 + torch.exp(-beta))
        g = g + s["dt_bias"]
        g = s["A"] * (g.clamp(min=0) + torch.log1p(torch.exp(-g.abs())))
    q = q * c["dk"] ** -0.5
    if s["lens"] is not None:           # a step of no rate and no decay leaves the state as it is
        on = (torch.arange(t, device=DEVICE) < s["lens"][:, None])[:, :, None]
        beta, g = torch.where(on, beta, 0.0), torch.where(on, g, 0.0)
    # [batch heads, chunks, steps of a chunk, ...]
    n = min(CHUNK, t)
    chunks = (t + n - 1) // n

    def cut(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, chunks * n - t))
        return x.transpose(1, 2).unflatten(2, (chunks, n)).flatten(0, 1)

    each = h // c["key_heads"]
    q, k = cut(q.repeat_interleave(each, 2)), cut(k.repeat_interleave(each, 2))
    v, beta, g = cut(v), cut(beta)[..., None], cut(g)
    # sums of decays, in 64 bits, where differences of far sums are taken
    total = g.double().cumsum(2)
    decay = torch.exp((total[..., :, None] - total[..., None, :]).float())
    below = torch.ones(n, n, device=DEVICE, dtype=torch.bool).tril(-1)
    apart = torch.where(below, decay * (k @ k.transpose(2, 3)) * beta, 0.0)
    # (1 + apart)^-1 as a product over doubled powers, in 64 bits: its terms
    # exceed their sum by far where keys are alike
    power = -apart.double()
    inverse = torch.eye(n, device=DEVICE, dtype=torch.float64) + power
    span = 2
    while span < n:
        power = power @ power
        inverse = inverse + inverse @ power
        span *= 2
    inverse = inverse.float()
    scores = torch.where(below | torch.eye(n, device=DEVICE, dtype=torch.bool),
                         decay * (q @ k.transpose(2, 3)), 0.0)
    since = torch.exp(total.float())[..., None]                   # decays from the chunk's start
    until = torch.exp((total[..., -1:] - total).float())[..., None]    # and to its end
    own_part = inverse @ (beta * v)
    reads, queries, writes = inverse @ (beta * since * k), since * q, (until * k).transpose(2, 3).contiguous()
    S = s["state"].flatten(0, 1) if s["state"] is not None else v.new_zeros(b * h, c["dk"], dv)
    outs = []
    for i in range(chunks):
        u = own_part[:, i] - reads[:, i] @ S
        outs.append(queries[:, i] @ S + scores[:, i] @ u)
        S = since[:, i, -1:] * S + writes[:, i] @ u
    o = torch.stack(outs, 1).flatten(1, 2)[:, :t].unflatten(0, (b, h)).transpose(1, 2)
    if s["lens"] is not None:
        o = torch.where(on[..., None], o, 0.0)
    return {"o": o.to(s["v"].dtype).contiguous(), "state": S.unflatten(0, (b, h))}


def _plain_norm(c, s):
    x = s["x"].float()
    gate = None
    if s["z"] is not None:
        z = s["z"].float()
        gate = z / (1 + torch.exp(-z))
    if c["gate"] == "before":
        x = x * gate
    y = x * torch.rsqrt((x * x).mean(2, keepdim=True) + NORM_EPS) * s["weight"]
    if c["gate"] == "after":
        y = y * gate
    return {"y": y.to(s["x"].dtype)}


def _plain_beam(c, s):
    b, n, v, keep = c["batch"], c["beams"], c["vocab"], c["keep"]
    x = s["logits"].float()
    most = x.amax(2, keepdim=True)
    # in 64 bits: candidates of unlike beams next to each other
    lse = most.double() + torch.log(torch.exp(x.double() - most).sum(2, keepdim=True))
    base = s["scores"].double()[..., None] - lse
    alive = torch.isfinite(base)
    ids = torch.arange(v, device=DEVICE)
    if s["finished"] is not None:
        ended = s["finished"][..., None]
        alive = alive & ~ended
        x = torch.where(alive, x, (ended & (ids == EOS)).float())
    else:
        x = torch.where(alive, x, 0.0)
    # one whole number for each value that orders by the value, then by the lower index
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 20) - ids
    best = torch.topk(key, min(keep, v), 2).indices
    value = torch.where(alive, base + x.gather(2, best), -math.inf)
    if s["finished"] is not None:
        mine = s["scores"].double()[..., None]
        value = torch.where(ended & (best == EOS) & torch.isfinite(mine), mine, value)
    value, at = torch.sort(value.flatten(1), dim=1, descending=True, stable=True)
    at = at[:, :keep]
    return {"scores": value[:, :keep].float(), "tokens": best.flatten(1).gather(1, at).int(),
            "parents": (at // best.shape[2]).int()}


def _plain_reorder(c, s):
    first = torch.arange(c["batch"], device=DEVICE, dtype=torch.int32)[:, None] * c["beams"]
    rows = (first + s["parents"]).flatten()
    return {"states": [x.index_select(s["dim"], rows) for x in s["states"]]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "delta":
        b, t, g, h, dk, dv = (case[k] for k in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
        moved = b * t * (2 * g * dk + 2 * h * dv) * size + b * t * 2 * h * (size if case["raw"] else 4)
        moved += b * h * dk * dv * 4 * (2 if case["state"] else 1)
        return {"bytes": moved, "flops": b * t * h * dk * dv * 7}
    if case["op"] == "norm":
        r, g, n = case["rows"], case["groups"], case["dim"]
        return {"bytes": r * g * n * size * (2 if case["gate"] == "none" else 3) + n * 4 * (1 if case["shared"] else g),
                "flops": r * g * n * (4 if case["gate"] == "none" else 8)}
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        return {"bytes": rows * (case["vocab"] * size + 4) + case["batch"] * case["keep"] * 12,
                "flops": 3 * rows * case["vocab"]}
    b, n, k, d = case["batch"], case["beams"], case["keep"], case["dim"]
    row = case["layers"] * (4 * d * size if case["kind"] == "lstm"
                            else 3 * d * size + case["heads"] * case["dk"] ** 2 * 4)
    return {"bytes": b * (n + k) * row + 4 * b * k, "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "norm": _exact_norm, "beam": _exact_beam,
            "reorder": _exact_reorder}[case["op"]](case, s)


def _exact_delta(c, s):
    b, t, h, dk, dv = (c[k] for k in ("batch", "steps", "heads", "dk", "dv"))
    group = torch.arange(h, device=DEVICE) // (h // c["key_heads"])
    S = s["state"].double() if s["state"] is not None else torch.zeros(b, h, dk, dv, device=DEVICE,
                                                                       dtype=torch.float64)
    o = S.new_zeros(b, t, h, dv)
    for i in range(t):
        q, k, v = s["q"][:, i].double()[:, group], s["k"][:, i].double()[:, group], s["v"][:, i].double()
        rate, log_decay = s["beta"][:, i].double(), s["g"][:, i].double()
        if c["raw"]:
            q = q / torch.sqrt(q.square().sum(2, keepdim=True) + KEY_EPS)
            k = k / torch.sqrt(k.square().sum(2, keepdim=True) + KEY_EPS)
            rate = torch.sigmoid(rate)
            log_decay = s["A"].double() * torch.nn.functional.softplus(log_decay + s["dt_bias"].double(),
                                                                       threshold=50.0)
        new = torch.exp(log_decay)[..., None, None] * S
        u = rate[..., None] * (v - (new * k[..., None]).sum(2))
        new = new + k[..., None] * u[:, :, None]
        out = (new * q[..., None]).sum(2) / math.sqrt(dk)
        if s["lens"] is not None:
            on = i < s["lens"]
            out = torch.where(on[:, None, None], out, 0.0)
            new = torch.where(on[:, None, None, None], new, S)
        o[:, i], S = out, new
    return {"o": o, "state": S}


def _exact_norm(c, s):
    x = s["x"].double()
    gate = 1.0 if s["z"] is None else torch.nn.functional.silu(s["z"].double())
    if c["gate"] == "before":
        x, gate = x * gate, 1.0
    rms = (x.square().sum(2, keepdim=True) / c["dim"] + NORM_EPS).sqrt()
    return {"y": x / rms * s["weight"].double() * gate}


def _exact_beam(c, s):
    out = []
    for i in range(c["batch"]):
        value = s["scores"][i].double()[:, None] + torch.log_softmax(s["logits"][i].double(), 1)
        value = torch.where(torch.isfinite(value), value, -math.inf)
        if s["finished"] is not None:
            ended = s["finished"][i]
            value[ended] = -math.inf
            value[ended, EOS] = s["scores"][i].double()[ended]
        value, order = torch.sort(value.flatten(), descending=True, stable=True)
        order = order[:c["keep"]]
        out.append((value[:c["keep"]], (order % c["vocab"]).int(), (order // c["vocab"]).int()))
    return dict(zip(("scores", "tokens", "parents"), (torch.stack(v) for v in zip(*out))))


def _exact_reorder(c, s):
    def one(x):
        x = x.unflatten(s["dim"], (c["batch"], c["beams"])).movedim((s["dim"], s["dim"] + 1), (0, 1))
        x = torch.stack([x[i][s["parents"][i].long()] for i in range(c["batch"])])
        return x.movedim((0, 1), (s["dim"], s["dim"] + 1)).flatten(s["dim"], s["dim"] + 1).double()
    return {"states": [one(x) for x in s["states"]]}
