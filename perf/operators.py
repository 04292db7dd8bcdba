"""Measured cases of the selective-state language-model operators.

A layer of such a model projects its tokens with 8-bit weights, passes them
through a short causal convolution and a selective state space scan, and the
model's logits are scored: the log probability of given tokens, the entropy
and the most likely alternatives.  Every case is one call of one of these
operators, on the tensors a program has in hand at that point.

With ``own`` false the operators run in their plain form (elementary torch
operations in 32 bits, rounded once at the end); with ``own`` true through
the entry points of ``recurrent_nn_amd``.  ``exact`` is the definition in 64
bits, written apart from the plain form.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A long prompt of one request: x is the first half of the input
        # projection's rows, the other half is the gate.
        {"name": "conv_prompt", "op": "conv", "batch": 1, "steps": 8192, "dim": 4096, "taps": 4,
         "silu": True, "bias": True, "state": False, "ragged": False, "dtype": "bf16"},
        # One new token for each of 64 running requests: latency.
        {"name": "conv_step", "op": "conv", "batch": 64, "steps": 1, "dim": 4096, "taps": 4,
         "silu": True, "bias": True, "state": True, "ragged": False, "dtype": "bf16"},
        # The scan of a long prompt of one request.
        {"name": "scan_prompt", "op": "scan", "batch": 1, "steps": 8192, "dim": 4096, "states": 16,
         "groups": 1, "gate": True, "skip": True, "state": False, "ragged": False, "dtype": "bf16"},
        # A batch of chunks of unlike lengths that go on from earlier states,
        # in 32 bits, as an evaluation runs it.
        {"name": "scan_ragged", "op": "scan", "batch": 8, "steps": 1000, "dim": 1024, "states": 16,
         "groups": 1, "gate": False, "skip": True, "state": True, "ragged": True, "dtype": "f32"},
        # One new token for each of 64 running requests.
        {"name": "scan_step", "op": "scan", "batch": 64, "steps": 1, "dim": 4096, "states": 16,
         "groups": 1, "gate": True, "skip": True, "state": True, "ragged": False, "dtype": "bf16"},
        # Activations of a prompt rounded to 8 bits, one scale for each token.
        {"name": "quantize_prompt", "op": "quantize", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # A small odd matrix in 32 bits: a weight's rows rounded at load.
        {"name": "quantize_odd", "op": "quantize", "rows": 333, "cols": 2501, "dtype": "f32"},
        # The input projection of a prompt.
        {"name": "project_prompt", "op": "project", "rows": 8192, "cols": 2048, "outs": 8192,
         "bias": False, "dtype": "bf16"},
        # The same projection for the new tokens of four requests: reading
        # the weights is all there is.
        {"name": "project_step", "op": "project", "rows": 4, "cols": 2048, "outs": 8192,
         "bias": False, "dtype": "bf16"},
        # A ragged batch of tokens through an odd-sized layer.
        {"name": "project_odd", "op": "project", "rows": 777, "cols": 1500, "outs": 2101,
         "bias": True, "dtype": "f16"},
        # Scoring every token of a prompt, with 20 alternatives each.
        {"name": "scores_prompt", "op": "scores", "rows": 1024, "vocab": 131072, "top": 20,
         "masked": False, "dtype": "bf16"},
        # The scores of the tokens just sampled for four requests, part of
        # the vocabulary masked out by a grammar.
        {"name": "scores_step", "op": "scores", "rows": 4, "vocab": 100001, "top": 8,
         "masked": True, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "quantize", "project", "project", "scores"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("conv", "scan"):
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.6:                    # whole 16-byte rows, as most models have them
            dim = max(64, dim // 64 * 64)
        batch = _log(rng, 1, 128)
        steps = 1 if rng.random() < 0.3 else _log(rng, 2, 8192)
        carry = steps == 1 or rng.random() < 0.5
        ragged = batch > 1 and steps > 1 and rng.random() < 0.5
        if op == "conv":
            most = 8192 * 4096
            steps = max(1, min(steps, most // (batch * dim)))
            return {"op": op, "batch": batch, "steps": steps, "dim": dim,
                    "taps": rng.choice([2, 3, 4, 4, 4, 5, 8]), "silu": rng.random() < 0.8,
                    "bias": rng.random() < 0.8, "state": carry, "ragged": ragged, "dtype": dtype}
        states = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
        groups = rng.choice([1, 1, 1, 2, 4])
        dim = max(groups, dim // groups * groups)
        most = 8192 * 4096 * 16
        steps = max(1, min(steps, most // (batch * dim * states)))
        return {"op": op, "batch": batch, "steps": steps, "dim": dim, "states": states,
                "groups": groups, "gate": rng.random() < 0.7, "skip": rng.random() < 0.8,
                "state": carry, "ragged": ragged, "dtype": dtype}
    if op == "quantize":
        cols = _log(rng, 16, 16384)
        return {"op": op, "rows": min(_log(rng, 1, 16384), 8192 * 4096 // cols), "cols": cols,
                "dtype": dtype}
    if op == "project":
        rows, cols, outs = _log(rng, 1, 8192), _log(rng, 32, 8192), _log(rng, 32, 16384)
        if rng.random() < 0.5:
            cols, outs = max(64, cols // 64 * 64), max(64, outs // 64 * 64)
        rows = max(1, min(rows, 8192 * 2048 * 8192 // (cols * outs)))
        return {"op": op, "rows": rows, "cols": cols, "outs": outs, "bias": rng.random() < 0.5,
                "dtype": dtype}
    vocab = _log(rng, 1000, 262144)
    rows = max(1, min(_log(rng, 1, 4096), 1024 * 131072 // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "top": rng.choice([0, 1, 5, 8, 20, 32]),
            "masked": rng.random() < 0.4, "dtype": dtype}


def _lengths(case, gen):
    """Lengths of the rows of a batch: at least one full row, and one of no
    steps where there are three rows or more."""
    n = torch.randint(1, case["steps"] + 1, (case["batch"],), generator=gen, device=DEVICE,
                      dtype=torch.int32)
    n[0] = case["steps"]
    if case["batch"] > 2:
        n[-1] = 0
    return n


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE, dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "conv":
        b, t, d, k = case["batch"], case["steps"], case["dim"], case["taps"]
        s["x"] = normal(b, t, 2 * d)[:, :, :d]        # rows of the input projection: [x, gate]
        s["weight"] = (uniform(d, k) * 2 - 1) / math.sqrt(k)
        s["bias"] = (uniform(d) * 2 - 1) / math.sqrt(k) if case["bias"] else None
        s["state"] = normal(b, k - 1, d) if case["state"] else None
        s["lens"] = _lengths(case, gen) if case["ragged"] else None
    elif case["op"] == "scan":
        b, t, d, n, g = (case[k] for k in ("batch", "steps", "dim", "states", "groups"))
        s["x"] = torch.nn.functional.silu(normal(b, t, d, dtype=torch.float32)).to(dt)
        s["dt"] = (normal(b, t, d, dtype=torch.float32) * 0.5).to(dt)
        # rows of the projection that gives B and C, behind the low-rank step sizes
        low = 16
        proj = normal(b, t, low + 2 * g * n)
        s["B"] = proj[:, :, low:low + g * n].unflatten(2, (g, n))
        s["C"] = proj[:, :, low + g * n:].unflatten(2, (g, n))
        s["A"] = -(torch.arange(1, n + 1, device=DEVICE, dtype=torch.float32) *
                   (0.8 + 0.4 * uniform(d, n)))
        size = torch.exp(uniform(d) * math.log(100.0) + math.log(1e-3))   # step sizes 0.001 to 0.1
        s["dt_bias"] = size + torch.log(-torch.expm1(-size))
        s["D"] = 0.5 + uniform(d) if case["skip"] else None
        s["z"] = normal(b, t, 2 * d)[:, :, d:] if case["gate"] else None
        s["state"] = normal(b, d, n, dtype=torch.float32) if case["state"] else None
        s["lens"] = _lengths(case, gen) if case["ragged"] else None
    elif case["op"] == "quantize":
        # activations with a few large channels
        s["x"] = (normal(case["rows"], case["cols"], dtype=torch.float32) *
                  torch.exp(normal(case["cols"], dtype=torch.float32))).to(dt)
    elif case["op"] == "project":
        m, k, n = case["rows"], case["cols"], case["outs"]
        s["x"] = (normal(m, k, dtype=torch.float32) *
                  torch.exp(0.5 * normal(k, dtype=torch.float32))).to(dt)
        # 8-bit weights, rows 16 bytes aligned, one scale for each output channel
        w = torch.zeros(n, (k + 15) // 16 * 16, device=DEVICE, dtype=torch.int8)
        w[:, :k] = torch.randn(n, k, generator=gen, device=DEVICE).mul_(38.0).round_().clamp_(-127, 127)
        s["w"] = w[:, :k]
        s["w_scale"] = (0.5 + uniform(n)) / (38.0 * math.sqrt(k))
        s["bias"] = uniform(n) - 0.5 if case["bias"] else None
    else:
        r, v = case["rows"], case["vocab"]
        logits = 2.5 * torch.randn(r, v, generator=gen, device=DEVICE)
        # the tokens: drawn from the distribution itself (random numbers are inputs here)
        noise = -torch.log(-torch.log(uniform(r, v).clamp_(1e-20, 1 - 1e-7)))
        if case["masked"]:
            logits.masked_fill_(uniform(r, v) < 0.5, -math.inf)
        logits = logits.to(dt)
        s["tokens"] = noise.add_(logits).argmax(1)
        s["logits"] = logits
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"conv": _plain_conv, "scan": _plain_scan, "quantize": _plain_quantize,
            "project": _plain_project, "scores": _plain_scores}[c["op"]](c, state)


def _own(c, s):
    import recurrent_nn_amd as ra
    if c["op"] == "conv":
        y, window = ra.causal_conv(s["x"], s["weight"], s["bias"], silu=c["silu"], state=s["state"],
                                   sequence_lens=s["lens"])
        return {"y": y, "state": window}
    if c["op"] == "scan":
        y, h = ra.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], dt_softplus=True, state=s["state"],
                                 sequence_lens=s["lens"])
        return {"y": y, "state": h}
    if c["op"] == "quantize":
        q, scale = ra.quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    if c["op"] == "project":
        return {"y": ra.quant_project(s["x"], s["w"], s["w_scale"], bias=s["bias"])}
    got = ra.token_scores(s["logits"], s["tokens"], top=c["top"])
    return {"logprob": got.logprob, "entropy": got.entropy, "rank": got.rank,
            "top_logprobs": got.top_logprobs, "top_ids": got.top_ids}


def _valid(c, s):
    """[batch, steps, 1]: the positions before each row's length."""
    return (torch.arange(c["steps"], device=DEVICE) < s["lens"][:, None])[:, :, None]


def _plain_conv(c, s):
    x, k = s["x"], c["taps"]
    before = s["state"] if s["state"] is not None else x.new_zeros(c["batch"], k - 1, c["dim"])
    rows = torch.cat([before, x], 1)
    y = (rows.float().unfold(1, k, 1) * s["weight"]).sum(-1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["silu"]:
        y = y / (1 + torch.exp(-y))
    if s["lens"] is None:
        return {"y": y.to(x.dtype), "state": rows[:, c["steps"]:].contiguous()}
    y = torch.where(_valid(c, s), y, 0.0)
    at = s["lens"].long()[:, None] + torch.arange(k - 1, device=DEVICE)
    window = rows.gather(1, at[:, :, None].expand(-1, -1, c["dim"]))
    return {"y": y.to(x.dtype), "state": window}


def _plain_scan(c, s):
    x = s["x"].float()
    step = s["dt"].float() + s["dt_bias"]
    step = step.clamp(min=0) + torch.log1p(torch.exp(-step.abs()))
    if s["lens"] is not None:
        step = torch.where(_valid(c, s), step, 0.0)     # a step of no size leaves the state as it is
    each = c["dim"] // c["groups"]
    B = s["B"].float().repeat_interleave(each, 2)
    C = s["C"].float().repeat_interleave(each, 2)
    a = torch.exp(step[..., None] * s["A"])
    h = (step * x)[..., None] * B
    if s["state"] is not None:
        h[:, 0] += a[:, 0] * s["state"]
    # h[t] = a[t] h[t-1] + h[t] for all steps, by doubling the span that each position has seen
    span = 1
    while span < c["steps"]:
        h[:, span:] += a[:, span:] * h[:, :-span]
        a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    last = h[:, -1].clone()
    y = (h * C).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    if s["lens"] is not None:
        y = torch.where(_valid(c, s), y, 0.0)
    return {"y": y.to(s["x"].dtype), "state": last}


def _quantized(x):
    """Rows to 8 bits: r = 127 / max|x| in binary32, q = x r rounded to the
    nearest even, and the scale max|x| / 127."""
    x = x.float()
    most = x.abs().amax(1, keepdim=True)
    full = torch.full_like(most, 127.0)      # a tensor: a number would be divided by its reciprocal
    return torch.round(x * (full / most)), most / full


def _plain_quantize(c, s):
    q, scale = _quantized(s["x"])
    return {"q": q.to(torch.int8), "scale": scale[:, 0]}


def _plain_project(c, s):
    q, scale = _quantized(s["x"])
    y = (q @ s["w"].float().t()) * scale * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype)}


def _plain_scores(c, s):
    x = s["logits"].float()
    token = s["tokens"][:, None]
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total)
    below = torch.where(e > 0, x - most, 0.0)
    entropy = lse - (e * below).sum(1, keepdim=True) / total
    mine = x.gather(1, token)
    ids = torch.arange(c["vocab"], device=DEVICE)
    rank = (x > mine).sum(1) + ((x == mine) & (ids < token)).sum(1)
    # one whole number for each value that orders by the value, then by the lower index
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 20) - ids
    top = torch.topk(key, c["top"], 1).indices
    return {"logprob": (mine - most - lse)[:, 0], "entropy": entropy[:, 0],
            "rank": rank.to(torch.int32), "top_logprobs": x.gather(1, top) - most - lse,
            "top_ids": top.to(torch.int32)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "conv":
        b, t, d, k = case["batch"], case["steps"], case["dim"], case["taps"]
        moved = 2 * b * t * d * size + d * (k + 1) * 4 + b * d * (k - 1) * size * (2 if case["state"] else 1)
        return {"bytes": moved, "flops": b * t * d * (2 * k + 4)}
    if case["op"] == "scan":
        b, t, d, n, g = (case[k] for k in ("batch", "steps", "dim", "states", "groups"))
        moved = b * t * size * (d * (4 if case["gate"] else 3) + 2 * g * n)
        moved += b * d * n * 4 * (2 if case["state"] else 1) + d * (n + 2) * 4
        return {"bytes": moved, "flops": b * t * d * (7 * n + 8)}
    if case["op"] == "quantize":
        r, k = case["rows"], case["cols"]
        return {"bytes": r * k * (size + 1) + 4 * r, "flops": 3 * r * k}
    if case["op"] == "project":
        m, k, n = case["rows"], case["cols"], case["outs"]
        return {"bytes": m * k * size + n * k + m * n * size + 8 * n, "flops": 2 * m * k * n}
    r, v = case["rows"], case["vocab"]
    return {"bytes": r * v * size + r * (20 + 8 * case["top"]), "flops": 6 * r * v}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "quantize": _exact_quantize,
            "project": _exact_project, "scores": _exact_scores}[case["op"]](case, s)


def _exact_conv(c, s):
    b, t, d, k = c["batch"], c["steps"], c["dim"], c["taps"]
    x = s["x"].double()
    past = s["state"].double() if s["state"] is not None else x.new_zeros(b, k - 1, d)
    w = s["weight"].double()
    y = x.new_zeros(b, t, d)
    for j in range(k):                        # tap j reaches back k - 1 - j steps
        back = k - 1 - j
        seen = min(back, t)
        y[:, back:] += w[:, j] * x[:, :t - back] if back < t else 0
        y[:, :seen] += w[:, j] * past[:, k - 1 - back:k - 1 - back + seen]
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["silu"]:
        y *= torch.sigmoid(y)
    window = x.new_zeros(b, k - 1, d)
    for i in range(b):
        n = t if s["lens"] is None else int(s["lens"][i])
        y[i, n:] = 0
        kept = min(n, k - 1)
        window[i, :k - 1 - kept] = past[i, kept:]
        if kept:
            window[i, k - 1 - kept:] = x[i, n - kept:n]
    return {"y": y, "state": window}


def _exact_scan(c, s):
    b, t, d, n = (c[k] for k in ("batch", "steps", "dim", "states"))
    group = torch.arange(d, device=DEVICE) // (d // c["groups"])
    A, bias = s["A"].double(), s["dt_bias"].double()
    h = s["state"].double() if s["state"] is not None else A.new_zeros(b, d, n)
    lens = torch.full((b,), t, device=DEVICE) if s["lens"] is None else s["lens"]
    y = A.new_zeros(b, t, d)
    for i in range(t):
        x = s["x"][:, i].double()
        step = torch.nn.functional.softplus(s["dt"][:, i].double() + bias, threshold=50.0)
        new = torch.exp(step[:, :, None] * A) * h
        new += (step * x)[:, :, None] * s["B"][:, i].double()[:, group]
        out = (new * s["C"][:, i].double()[:, group]).sum(2)
        if s["D"] is not None:
            out = out + s["D"].double() * x
        if s["z"] is not None:
            out = out * torch.nn.functional.silu(s["z"][:, i].double())
        if s["lens"] is None:
            y[:, i], h = out, new
        else:
            on = i < lens
            y[:, i] = torch.where(on[:, None], out, 0.0)
            h = torch.where(on[:, None, None], new, h)
    return {"y": y, "state": h}


def _single(v):
    """A 64-bit value rounded to binary32, where the definition rounds."""
    return v.to(torch.float32).double()


def _exact_rows(x):
    x = x.double()
    most = torch.maximum(x.max(1).values, -x.min(1).values)[:, None]
    full = torch.full_like(most, 127.0)
    return torch.round(_single(x * _single(full / most))), _single(most / full)


def _exact_quantize(c, s):
    q, scale = _exact_rows(s["x"])
    return {"q": q.to(torch.int8), "scale": scale[:, 0]}


def _exact_project(c, s):
    q, scale = _exact_rows(s["x"])
    y = torch.mm(q, s["w"].double().t().contiguous()) * scale * s["w_scale"].double()
    return {"y": y if s["bias"] is None else y + s["bias"].double()}


def _exact_scores(c, s):
    top, out = c["top"], []
    for lo in range(0, c["rows"], 256):
        x, token = s["logits"][lo:lo + 256].double(), s["tokens"][lo:lo + 256, None]
        logp = torch.log_softmax(x, 1)
        p = torch.exp(logp)
        entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        rank = (order == token).int().argmax(1)
        out.append((logp.gather(1, token)[:, 0], entropy, rank.int(),
                    logp.gather(1, order[:, :top]), order[:, :top].int()))
    return dict(zip(("logprob", "entropy", "rank", "top_logprobs", "top_ids"),
                    (torch.cat(v) for v in zip(*out))))
