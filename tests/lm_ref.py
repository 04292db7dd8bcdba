"""Plain 64-bit definitions of the language-model operators on the CPU, with
a bound on the error of a float32 evaluation that each test compares against.

U is half a step of float32 (2^-24), relative: what one rounded operation is
off by at most.  The hardware's exp2, log2 and reciprocal are taken as one step
(2 U).  Every bound counts roundings along the written formula and doubles
them, since a kernel may associate sums and products in another order.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
SMALLEST = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def d(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def stored(y, err, dtype):
    """`err` with the rounding to `dtype` added."""
    return err * (1 + 2 * HALF_STEP[dtype]) + np.abs(y) * HALF_STEP[dtype] + SMALLEST[dtype]


def silu_err(v, err):
    """silu(v) and its error, for v off by err: |silu'| <= 1.1; the exponent
    v log2 e is off by 2 U |v| and exp2, 1 +, reciprocal and product add 8 U."""
    y = v * sigmoid(v)
    return y, 1.1 * err + np.abs(y) * (2 * np.abs(v) + 12) * U


def conv(x, weight, bias, silu, state, lens):
    """(y, error of y, window) as float64 arrays."""
    dtype = x.dtype
    x, w, bias = d(x), d(weight), d(bias)
    b, t, c = x.shape
    k = w.shape[1]
    past = d(state) if state is not None else np.zeros((b, k - 1, c))
    y, err, win = np.zeros((b, t, c)), np.zeros((b, t, c)), np.zeros((b, k - 1, c))
    for i in range(b):
        n = t if lens is None else min(max(int(lens[i]), 0), t)
        rows = np.concatenate([past[i], x[i, :n]])
        for s in range(n):
            terms = rows[s:s + k] * w.T
            v = terms.sum(0) + (0 if bias is None else bias)
            e = 2 * (k + 1) * U * (np.abs(terms).sum(0) + (0 if bias is None else np.abs(bias)))
            y[i, s], err[i, s] = silu_err(v, e) if silu else (v, e)
        err[i, :n] = stored(y[i, :n], err[i, :n], dtype)
        win[i] = rows[n:n + k - 1]
    return y, err, win


def scan(x, dt, A, B, C, D, z, dt_bias, softplus, state, lens):
    """(y, error of y, state, error of the state)."""
    dtype = x.dtype
    x, dt, A, B, C, D, z, dt_bias = (d(v) for v in (x, dt, A, B, C, D, z, dt_bias))
    b, t, c = x.shape
    n = A.shape[1]
    if B.ndim == 3:
        B, C = B[:, :, None], C[:, :, None]
    per = c // B.shape[2]
    h = d(state) if state is not None else np.zeros((b, c, n))
    h = h.copy()
    e = np.zeros_like(h)
    y, err = np.zeros((b, t, c)), np.zeros((b, t, c))
    for i in range(b):
        steps = t if lens is None else min(max(int(lens[i]), 0), t)
        for s in range(steps):
            v = dt[i, s] + (0 if dt_bias is None else dt_bias)
            # the sum's rounding and (softplus) the exponent and the series
            off = 2 * U * (np.abs(dt[i, s]) + (0 if dt_bias is None else np.abs(dt_bias)))
            step = np.logaddexp(0, v) if softplus else v
            serr = sigmoid(v) * off + np.abs(step) * (2 * np.abs(v) + 24) * U if softplus else off
            Bt, Ct = np.repeat(B[i, s], per, 0), np.repeat(C[i, s], per, 0)
            arg = step[:, None] * A
            with np.errstate(over="ignore"):
                a = np.exp(arg)
            aerr = serr[:, None] * np.abs(A) + 4 * U * np.abs(arg) + 2 * U
            u = (step * x[i, s])[:, None] * Bt
            uerr = (serr * np.abs(x[i, s]))[:, None] * np.abs(Bt) + 6 * U * np.abs(u)
            # a state may be formed from a run's local state and the run's decay
            e[i] = a * e[i] + np.abs(a * h[i]) * (2 * aerr + 4 * U) + uerr
            h[i] = a * h[i] + u
            e[i] += 2 * U * np.abs(h[i])
            o = (Ct * h[i]).sum(1)
            oe = (np.abs(Ct) * e[i]).sum(1) + 2 * (n + 2) * U * np.abs(Ct * h[i]).sum(1)
            if D is not None:
                oe += 4 * U * (np.abs(D * x[i, s]) + np.abs(o))
                o = o + D * x[i, s]
            if z is not None:
                gate, ge = silu_err(z[i, s], 0)
                oe = oe * np.abs(gate) + np.abs(o) * ge + 4 * U * np.abs(o * gate)
                o = o * gate
            y[i, s], err[i, s] = o, stored(o, oe, dtype)
    return y, err, h, e + 2.0 ** -126


def quantize(x):
    """(q, scale), in float32 as the definition says: bit for bit."""
    x = x.detach().cpu().float().numpy()
    q = np.zeros(x.shape, np.int8)
    scale = np.zeros(x.shape[0], np.float32)
    for i, row in enumerate(x):
        if not np.isfinite(row).all():
            scale[i] = np.nan
            continue
        most = np.float32(np.abs(row).max()) if row.size else np.float32(0)
        if most < np.float32(2.0 ** -100):
            continue
        r = np.float32(127) / most
        q[i] = np.rint(row * r).astype(np.int8)
        scale[i] = most / np.float32(127)
    return q, scale


def project(q, scale, w, w_scale, bias, dtype):
    """(y, error): the sum is exact, three roundings and bias follow."""
    total = q.astype(np.float64) @ d(w).T
    y = total * scale.astype(np.float64)[:, None] * d(w_scale)
    err = 4 * U * np.abs(y)
    if bias is not None:
        y = y + d(bias)
        err = err + 2 * U * np.abs(y)
    return y, stored(y, 2 * err, dtype)


def order(x):
    """Indices of a row by value, larger first (NaN before all), equal ones
    by index."""
    x = np.where(np.isnan(x), np.inf, x), np.isnan(x)
    return np.lexsort((np.arange(x[0].size), -x[0], ~x[1]))


def scores(logits, tokens, top):
    """dict of logprob, entropy, rank, top_logprobs, top_ids, and `err`, a
    bound on every log probability and (err_entropy) on the entropy."""
    x = d(logits)
    rows, v = x.shape
    out = {"logprob": np.full(rows, np.nan), "entropy": np.full(rows, np.nan),
           "rank": np.full(rows, -1, np.int64), "top_logprobs": np.full((rows, top), -np.inf),
           "top_ids": np.full((rows, top), -1, np.int64), "err": np.zeros(rows),
           "err_entropy": np.zeros(rows)}
    for i in range(rows):
        at = order(x[i])
        keep = at[:top]
        out["top_ids"][i, :len(keep)] = keep
        with np.errstate(all="ignore"):
            below = x[i] - x[i].max()
            e = np.exp(below)
            total = e.sum()
            lse = np.log(total)
            logp = below - lse
            p = e / total
            out["entropy"][i] = -np.where(p > 0, p * logp, np.where(np.isnan(p), np.nan, 0)).sum()
        out["top_logprobs"][i, :len(keep)] = logp[keep]
        token = None if tokens is None else int(tokens[i])
        if token is not None and 0 <= token < v:
            out["logprob"][i] = logp[token]
            out["rank"][i] = int(np.nonzero(at == token)[0][0])
        # each exponential: the difference and the product round, exp2 is one
        # step; sums of v positive terms in at least 64 strands
        with np.errstate(all="ignore"):
            rel = np.nansum(p * 6 * U * np.where(p > 0, np.abs(below), 0)) + (v / 64 + 64) * 2 * U
            out["err"][i] = rel + 8 * U * (1 + abs(lse))
            out["err_entropy"][i] = 2 * rel * (1 + abs(out["entropy"][i])) + 16 * U * (1 + abs(lse))
    return out


def assert_close(got, want, err, what):
    """|got - want| <= err where want is finite, the same value elsewhere."""
    got = d(got) if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    rest = ~fine & ~np.isnan(want)
    assert np.array_equal(got[rest], want[rest]), f"{what}: infinities differ"
    err = np.broadcast_to(err, want.shape)
    over = np.abs(got - want)[fine] - err[fine]
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: off by {np.abs(got - want)[fine].max():.3e}, {over.max():.3e} more than allowed"
