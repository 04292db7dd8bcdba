"""Operators of a delta-rule language model, and of decoding with several beams,
on torch tensors: the thin binding of rnn_delta_run, rnn_gated_norm,
rnn_beam_select and rnn_reorder_states (include/recurrent_nn_amd.h has their
definitions).

As in :mod:`recurrent_nn_amd.lm`: forward only (a tensor that requires a
gradient is refused while gradients are recorded); tensors live on one HIP
device; the work goes to ``stream`` (default: torch's current stream of that
device) and nothing waits for it; what a call returns is new unless ``out`` /
``state_out`` supply it; ValueError for tensors of the wrong kind, RNNError for
what the library refuses.  A plain call is checked and made by the compiled
module _binding (csrc/binding_delta.cpp) in one step; what it does not take
goes the way below, with the same steps.
"""
from __future__ import annotations

import ctypes
from typing import List, NamedTuple, Optional, Sequence, Union

import torch

from . import _check, _lib, lm
from ._lib import rnn_beam_desc, rnn_delta_desc, rnn_norm_desc, rnn_reorder_item
from .lm import _data, _done, _DTYPES, _expect, _lens, _no_gradient, _on, _ptr, _workspace

_ENTRIES = ("rnn_delta_workspace_size", "rnn_delta_run", "rnn_gated_norm", "rnn_beam_workspace_size",
            "rnn_beam_select", "rnn_reorder_states")
_bound = None


def _bind():
    """The compiled module, with the entry points of the loaded library."""
    global _bound
    lib, compiled = _lib.load(), lm._bind()
    compiled.bind_delta(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES])
    _bound = compiled
    return _bound


def gated_delta(q, k, v, beta, g=None, A=None, dt_bias=None, beta_sigmoid: bool = False,
                normalize: bool = False, scale: Optional[float] = None, state=None, sequence_lens=None,
                out=None, state_out=None, stream=None):
    """Gated delta rule: S = e^a S, u = b (v - S^T k), S = S + k u^T, o = scale S^T q.

    q, k [batch, steps, key_heads, key_dim] and v [batch, steps, heads,
    value_dim] of one type (last dimension contiguous, other strides free;
    head j reads key head j // (heads // key_heads)); beta and g [batch, steps,
    heads], both float32 or of v's type; A, dt_bias [heads] and state [batch,
    heads, key_dim, value_dim] float32; sequence_lens as in
    :func:`recurrent_nn_amd.causal_conv`.  b = beta, or its sigmoid with
    ``beta_sigmoid``; a = g (None: 0), or A softplus(g + dt_bias) with ``A``, at
    most 0.  ``normalize`` divides q and k by sqrt(sum x^2 + 1e-6).  scale: None
    for key_dim ** -0.5.  Returns (o, state_out).  One new token: steps = 1.
    ``state_out`` may be ``state``.
    """
    if stream is None and getattr(q, "is_cuda", False):
        device = lm._device()
        r = (_bound or _bind()).delta(q, k, v, beta, g, A, dt_bias, beta_sigmoid, normalize, scale, state,
                                      sequence_lens, out, state_out, device, lm._raw_stream(device))
        if r is not None:
            return _done(r, "rnn_delta_run")
    _no_gradient(q=q, k=k, v=v, beta=beta, g=g, A=A, dt_bias=dt_bias, state=state, out=out,
                 state_out=state_out)
    lib = _lib.load()
    _data("q", q, 4)
    _data("v", v, 4)
    b, t, kh, dk = q.shape
    h, dv = v.shape[2:]
    if dk < 1:
        raise ValueError("q must have a column at least")
    _data("beta", beta, 3)
    if beta.dtype not in (torch.float32, v.dtype):
        raise ValueError("beta must be float32 or of v's type")
    for name, x, shape, kind in (("k", k, q.shape, q.dtype), ("v", v, (b, t, h, dv), q.dtype),
                                 ("beta", beta, (b, t, h), beta.dtype), ("g", g, (b, t, h), beta.dtype),
                                 ("out", out, v.shape, q.dtype)):
        if x is not None:
            _expect(name, x, shape, kind, q.device, dense=False)
    for name, x, shape in (("A", A, (h,)), ("dt_bias", dt_bias, (h,)), ("state", state, (b, h, dk, dv)),
                           ("state_out", state_out, (b, h, dk, dv))):
        if x is not None:
            _expect(name, x, shape, torch.float32, q.device)
    lens = _lens(sequence_lens, b, t, q.device)
    os = (t * h * dv, h * dv, dv) if out is None else out.stride()
    gs = (0, 0) if g is None else g.stride()
    desc = rnn_delta_desc(b, t, kh, h, dk, dv, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *os[:3],
                          *beta.stride()[:2], *gs[:2], _DTYPES[q.dtype], _DTYPES[beta.dtype],
                          bool(normalize), bool(beta_sigmoid), dk ** -0.5 if scale is None else scale)
    size = _workspace(lib.rnn_delta_workspace_size, desc)

    def call(s):
        o = q.new_empty((b, t, h, dv)) if out is None else out
        end = q.new_empty((b, h, dk, dv), dtype=torch.float32) if state_out is None else state_out
        ws = q.new_empty(size, dtype=torch.uint8) if size else None
        _check(lib.rnn_delta_run(ctypes.addressof(desc), s, _ptr(ws), size, q.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), beta.data_ptr(), _ptr(g), _ptr(A), _ptr(dt_bias), _ptr(state),
                                 _ptr(lens), o.data_ptr(), end.data_ptr()), "rnn_delta_run")
        return o, end

    return _on((q, k, v, beta, g, A, dt_bias, state, lens, out, state_out), stream, call)


def gated_norm(x, weight, z=None, gate_first: bool = False, eps: float = 1e-6, out=None, stream=None):
    """y = x / sqrt(mean x^2 + eps) * weight * silu(z) over each group of x.

    x, z [rows, groups, dim], or [rows, dim] for one group, of one type (last
    dimension contiguous, other strides free); weight [dim], shared by the
    groups, or [groups, dim], float32.  ``gate_first``: x silu(z) in the place
    of x, and no gate after.  ``out`` may be ``x`` or ``z``.
    """
    if stream is None and getattr(x, "is_cuda", False):
        device = lm._device()
        r = (_bound or _bind()).norm(x, weight, z, gate_first, eps, out, device, lm._raw_stream(device))
        if r is not None:
            return _done(r, "rnn_gated_norm")[0]
    _no_gradient(x=x, weight=weight, z=z, out=out)
    lib = _lib.load()
    _data("x", x, 2 if x.dim() == 2 else 3)
    rows, groups, dim = x.shape if x.dim() == 3 else (x.shape[0], 1, x.shape[1])
    for name, t in (("z", z), ("out", out)):
        if t is not None:
            _expect(name, t, x.shape, x.dtype, x.device, dense=False)
    _expect("weight", weight, (dim,) if weight.dim() == 1 else (groups, dim), torch.float32, x.device)

    def of(t):
        s = t.stride()
        return (s[0], s[1] if len(s) == 3 else 0)

    ys = (groups * dim, dim if x.dim() == 3 else 0) if out is None else of(out)
    desc = rnn_norm_desc(rows, groups, dim, *of(x), *((0, 0) if z is None else of(z)), *ys,
                         0 if weight.dim() == 1 else dim, _DTYPES[x.dtype], bool(gate_first), eps)

    def call(s):
        y = x.new_empty(x.shape) if out is None else out
        _check(lib.rnn_gated_norm(ctypes.addressof(desc), s, x.data_ptr(), weight.data_ptr(), _ptr(z),
                                  y.data_ptr()), "rnn_gated_norm")
        return y

    return _on((x, weight, z, out), stream, call)


class BeamChoice(NamedTuple):
    """What :func:`beam_select` chose, best first."""
    scores: torch.Tensor        # [batch, keep] float32
    tokens: torch.Tensor        # [batch, keep] int32
    parents: torch.Tensor       # [batch, keep] int32: the beam that each continues


def beam_select(logits, scores, keep: Optional[int] = None, finished=None, eos: Optional[int] = None,
                stream=None) -> BeamChoice:
    """The first ``keep`` continuations (default: as many as beams) of each
    request's beams by scores[b, i] + log softmax(logits[b, i])[token], equal
    ones in the order of beam and token.

    logits [batch, beams, vocab] float32, bfloat16 or float16 (last dimension
    contiguous, other strides free); scores [batch, beams] float32, -inf for a
    beam that is not there.  finished [batch, beams] bool (or uint8): such a
    beam is not continued, and stands by itself with the token ``eos`` and its
    score.  Where there are fewer candidates, the rest has score -inf and token
    and parent -1.
    """
    if stream is None and getattr(logits, "is_cuda", False):
        device = lm._device()
        r = (_bound or _bind()).beam(logits, scores, keep, finished, eos, device, lm._raw_stream(device))
        if r is not None:
            return BeamChoice._make(_done(r, "rnn_beam_select"))
    _no_gradient(logits=logits, scores=scores)
    lib = _lib.load()
    _data("logits", logits, 3)
    b, beams, vocab = logits.shape
    keep = beams if keep is None else int(keep)
    _expect("scores", scores, (b, beams), torch.float32, logits.device)
    if finished is not None:
        if eos is None:
            raise ValueError("finished beams need eos")
        _expect("finished", finished, (b, beams), torch.uint8 if finished.dtype == torch.uint8 else torch.bool,
                logits.device)
    desc = rnn_beam_desc(b, beams, vocab, logits.stride(0), logits.stride(1), _DTYPES[logits.dtype], keep,
                         0 if finished is None else int(eos))
    size = _workspace(lib.rnn_beam_workspace_size, desc)

    def call(s):
        ws = logits.new_empty(size, dtype=torch.uint8) if size else None
        value = logits.new_empty((b, keep), dtype=torch.float32)
        tokens, parents = (logits.new_empty((b, keep), dtype=torch.int32) for _ in range(2))
        _check(lib.rnn_beam_select(ctypes.addressof(desc), s, _ptr(ws), size, logits.data_ptr(),
                                   scores.data_ptr(), _ptr(finished), value.data_ptr(), tokens.data_ptr(),
                                   parents.data_ptr()), "rnn_beam_select")
        return BeamChoice(value, tokens, parents)

    return _on((logits, scores, finished), stream, call)


def reorder_states(states: Sequence[torch.Tensor], parents, dim: Union[int, Sequence[int]] = 0, out=None,
                   stream=None) -> List[torch.Tensor]:
    """States of beams in the order of a selection: row b keep + j of each new
    state is row b beams + parents[b, j] of the old one.

    states: contiguous tensors of any type with batch * beams rows along
    ``dim`` (one for all, or one for each); parents [batch, keep] int32 on the
    device (values outside [0, beams) are taken as the nearest end), as
    :func:`beam_select` gives them.  All tensors go in one launch for up to 32.
    ``out``: tensors for the results; a state's own (keep = beams) is reordered
    in place, and only rows that change are touched.  No result may lie on
    another state or result.
    """
    states = list(states)
    out = None if out is None else list(out)
    if stream is None and states and type(dim) is int and getattr(states[0], "is_cuda", False):
        device = lm._device()
        r = (_bound or _bind()).reorder(states, parents, dim, out, device, lm._raw_stream(device))
        if r is not None:
            return _done(r, "rnn_reorder_states")
    _no_gradient(**{f"states[{i}]": t for i, t in enumerate(states)},
                 **{f"out[{i}]": t for i, t in enumerate(out or ())})
    lib = _lib.load()
    if not isinstance(parents, torch.Tensor) or not parents.is_cuda or parents.dim() != 2:
        raise ValueError("parents must be a device tensor [batch, keep]")
    batch, keep = parents.shape
    device = parents.device
    _expect("parents", parents, (batch, keep), torch.int32, device)
    dims = [dim] * len(states) if isinstance(dim, int) else list(dim)
    if len(dims) != len(states) or (out is not None and len(out) != len(states)):
        raise ValueError("dim and out must have an entry for each state")
    beams, plan = 1, []
    for i, (x, d) in enumerate(zip(states, dims)):
        if not isinstance(x, torch.Tensor) or not x.is_cuda or x.device != device or not x.is_contiguous():
            raise ValueError(f"states[{i}] must be a contiguous tensor on {device}")
        if not -x.dim() <= d < x.dim():
            raise ValueError(f"states[{i}] has no dimension {d}")
        d %= x.dim()
        rows = x.shape[d]
        if batch and (rows % batch or (plan and rows != batch * beams)):
            raise ValueError(f"states[{i}] must have {'as many rows for each request' if plan else 'rows'} "
                             f"of {batch} requests along dimension {d}, not {rows} rows")
        if not batch and rows:
            raise ValueError(f"states[{i}] must have no rows, as parents")
        beams = rows // batch if batch else 1
        if beams < 1:
            raise ValueError(f"states[{i}] must have a beam for each request at least")
        shape = (*x.shape[:d], batch * keep, *x.shape[d + 1:])
        if out is not None:
            _expect(f"out[{i}]", out[i], shape, x.dtype, device)
        outer, inner = 1, x.element_size()
        for n in x.shape[:d]:
            outer *= n
        for n in x.shape[d + 1:]:
            inner *= n
        plan.append((shape, outer, inner))

    def call(s):
        new = [x.new_empty(p[0]) for x, p in zip(states, plan)] if out is None else out
        items = (rnn_reorder_item * max(1, len(plan)))(
            *[(_ptr(x), _ptr(y), p[1], p[2]) for x, y, p in zip(states, new, plan)])
        _check(lib.rnn_reorder_states(s, batch, beams, keep, _ptr(parents), ctypes.addressof(items),
                                      len(plan)), "rnn_reorder_states")
        return new

    return _on((parents, *states, *(out or ())), stream, call)
