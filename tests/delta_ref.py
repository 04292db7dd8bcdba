"""Plain 64-bit definitions of the delta-rule operators and of decoding with
several beams, on the CPU, with bounds on the error of a float32 evaluation.

The bounds count roundings (U = 2^-24 relative each) along the written sums and
double them.  For the delta rule they hold for steps taken one by one and for
chunks of 64 that solve a triangular system: within a chunk the corrections are
u = (1 + L)^-1 R, whose computed form is off by the errors of L and R through
|(1 + L)^-1|, and by the roundings of the inverse; what a chunk begins with is
off by E (a 2-norm for each column), and passes on through the steps' own maps
e^a (1 - b k k^T), of norm max(1, |1 - b |k|^2|) at most.
"""
import numpy as np
import torch

from tests.lm_ref import U, d, sigmoid, silu_err, stored

CHUNK = 64
KEY_EPS = 1e-6


def _gates(beta, g, A, dt_bias, beta_sigmoid):
    """(rate, its relative error), (log of the decay, its absolute error)."""
    rate, rate_err = beta, np.zeros_like(beta)
    if beta_sigmoid:
        rate, rate_err = sigmoid(beta), (np.abs(beta) + 8) * U
    if g is None:
        a, a_err = np.zeros_like(beta), np.zeros_like(beta)
    elif A is None:
        a, a_err = g, np.zeros_like(g)
    else:
        x = g + (0 if dt_bias is None else dt_bias)
        off = 2 * U * (np.abs(g) + (0 if dt_bias is None else np.abs(dt_bias)))
        a = A * np.logaddexp(0, x)
        a_err = np.abs(A) * sigmoid(x) * off + np.abs(a) * (2 * np.abs(x) + 16) * U
    inside = (a <= 0) & (a >= -104)
    return rate, rate_err, np.clip(a, -104, 0), np.where(inside, a_err, 0)


def delta(q, k, v, beta, g=None, A=None, dt_bias=None, beta_sigmoid=False, normalize=False, scale=None,
          state=None, lens=None):
    """(o, error of o, state, error of the state) as float64 arrays."""
    dtype = v.dtype
    q, k, v, beta, g, A, dt_bias = (d(x) for x in (q, k, v, beta, g, A, dt_bias))
    b, t, kh, dk = q.shape
    h, dv = v.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    S = np.zeros((b, h, dk, dv)) if state is None else d(state).copy()
    E = np.zeros((b, h, dv))
    o, err = np.zeros((b, t, h, dv)), np.zeros((b, t, h, dv))
    for i in range(b):
        n = t if lens is None else min(max(int(lens[i]), 0), t)
        rate, rate_err, a, a_err = _gates(beta[i, :n], None if g is None else g[i, :n], A, dt_bias,
                                          beta_sigmoid)
        qi, ki = q[i, :n], k[i, :n]
        if normalize:
            qi = qi / np.sqrt((qi ** 2).sum(-1, keepdims=True) + KEY_EPS)
            ki = ki / np.sqrt((ki ** 2).sum(-1, keepdims=True) + KEY_EPS)
        for j in range(h):
            at = j // (h // kh)
            for lo in range(0, n, CHUNK):
                s = slice(lo, min(lo + CHUNK, n))
                m = s.stop - lo
                qc, kc, vc, r = qi[s, at], ki[s, at], v[i, s, j], rate[s, j][:, None]
                G, D = np.cumsum(a[s, j]), np.exp(np.cumsum(a[s, j]))[:, None]
                # relative errors of the decay from the chunk's start (from step to
                # step: gap_err), and of a rate, the norms and a sum over dk
                sums = np.cumsum(a_err[s, j])
                De = (2 * sums + (4 * np.abs(G) + 8) * U)[:, None]
                gap_err = 2 * np.abs(sums[:, None] - sums[None]) + (4 * np.abs(G[:, None] - G[None]) + 8) * U
                one = rate_err[s, j][:, None] + (2 * dk + 24) * U
                S0 = S[i, j].copy()
                # the definition, step by step
                us = np.zeros((m, dv))
                for x in range(m):
                    S[i, j] *= np.exp(a[lo + x, j])
                    us[x] = r[x] * (vc[x] - kc[x] @ S[i, j])
                    S[i, j] += np.outer(kc[x], us[x])
                    o[i, lo + x, j] = scale * (qc[x] @ S[i, j])
                # the bound
                gap = np.where(np.tri(m, dtype=bool), np.exp(np.minimum(G[:, None] - G[None], 0)), 0)
                kq, kk = np.abs(qc) @ np.abs(kc).T, np.abs(kc) @ np.abs(kc).T
                norm_k, norm_q = (np.linalg.norm(x, axis=1)[:, None] for x in (kc, qc))
                L = np.tril(r * gap * (kc @ kc.T), -1)
                L_err = np.tril(np.abs(r) * gap * kk * (one + gap_err), -1)
                T = np.abs(np.linalg.inv(np.eye(m) + L))
                S0k, S0q = D * (np.abs(kc) @ np.abs(S0)), D * (np.abs(qc) @ np.abs(S0))
                R = np.abs(r) * (np.abs(vc) + S0k)
                u_err = T @ (np.abs(r) * (one * np.abs(vc) + (one + De) * S0k) + L_err @ np.abs(us)) + \
                    4 * CHUNK * U * (T @ ((np.eye(m) + np.abs(L)) @ (T @ R)))
                rho = np.cumprod(np.maximum(1, np.abs(1 - r[:, 0] * norm_k[:, 0] ** 2)))[:, None]
                back = rho.max() / rho                      # of an error that comes in later
                more = (CHUNK + 8) * U
                e = np.abs(scale) * (norm_q * D * rho * E[i, j] + (gap * kq) @ u_err +
                                     (gap * kq * (one + gap_err + more)) @ np.abs(us) +
                                     (one + De + more) * S0q)
                err[i, s, j] = stored(o[i, s, j], 2 * e, dtype)
                last, more = gap[-1][:, None], (4 * CHUNK + 16) * U
                E[i, j] = D[-1] * rho[-1] * E[i, j] + (last * norm_k * (
                    u_err + back * (one + gap_err[-1][:, None] + more) * np.abs(us))).sum(0) + \
                    (De[-1] + more) * D[-1] * rho[-1] * np.linalg.norm(S0, axis=0)
    return o, err, S, np.broadcast_to(2 * E[:, :, None], S.shape) + 2.0 ** -126


def norm(x, weight, z, gate_first, eps):
    """(y, error of y) for x [rows, groups, dim]."""
    dtype = x.dtype
    x, weight, z = d(x), d(weight), d(z)
    n = x.shape[-1]
    err = 0 * x
    gate, gate_err = (np.ones_like(x), 0 * x) if z is None else silu_err(z, 0)
    if gate_first:
        err = np.abs(x) * gate_err + 2 * U * np.abs(x * gate)
        x = x * gate
    mean = (x ** 2).mean(-1, keepdims=True) + eps
    # the sum of n squares; each off by 2 |x| err more
    mean_err = (2 * np.abs(x) * err).mean(-1, keepdims=True) + (n + 8) * U * mean
    y = x / np.sqrt(mean) * weight
    rel = 0.5 * mean_err / mean + 8 * U
    e = err / np.sqrt(mean) * np.abs(weight) + np.abs(y) * rel
    if z is not None and not gate_first:
        e = e * np.abs(gate) + np.abs(y) * gate_err + 2 * U * np.abs(y * gate)
        y = y * gate
    return y, stored(y, 2 * e, dtype)


def beam(logits, scores, keep, finished=None, eos=0):
    """(scores, tokens, parents): every candidate in order."""
    x, scores = d(logits), d(scores)
    b, n, v = x.shape
    out = np.full((b, keep), -np.inf), np.full((b, keep), -1), np.full((b, keep), -1)
    for i in range(b):
        value = np.full((n, v), -np.inf)
        for j in range(n):
            if not np.isfinite(scores[i, j]):
                continue
            if finished is not None and bool(finished[i, j]):
                value[j, eos] = scores[i, j]
                continue
            row = x[i, j]
            if np.isnan(row).any() or np.isposinf(row).any() or np.isneginf(row).all():
                continue
            m = row.max()
            value[j] = scores[i, j] - (m + np.log(np.exp(row - m).sum())) + row
        order = np.argsort(-value.ravel(), kind="stable")[:keep]
        for o, w in zip(out, (value.ravel()[order], order % v, order // v)):
            o[i, :len(order)] = w
    return out


def reorder(x, parents, dim):
    """The rows of x in the order of parents [batch, keep]."""
    b, keep = parents.shape
    beams = x.shape[dim] // b
    rows = (torch.arange(b)[:, None] * beams + parents.long().clamp(0, beams - 1)).flatten()
    return x.index_select(dim, rows)
