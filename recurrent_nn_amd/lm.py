"""Operators of a selective-state language model on torch tensors: the thin
binding of rnn_conv_run, rnn_scan_run, rnn_quantize_rows, rnn_quant_project
and rnn_token_scores (include/recurrent_nn_amd.h has their definitions).

Forward only: nothing is recorded for gradients, and while they are recorded a
tensor that requires one is refused (call under torch.no_grad(), or pass what
detach() gives).  Tensors live on one HIP device; the work goes to ``stream``
(default: torch's current stream of that device) and nothing waits for it.
What a call returns is new unless ``out`` / ``state_out`` supply it.  ValueError
for tensors of the wrong kind, RNNError for what the library refuses.

A call on the current device's current stream, with every tensor as it should
be, is checked and made by the compiled module _binding (csrc/binding.cpp) in
one step.  What it does not take (it returns None and has done nothing) goes
the way below, with the same steps.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _lib
from ._lib import (RNN_DTYPE_BF16, RNN_DTYPE_F16, RNN_DTYPE_F32, RNN_DTYPE_I8, rnn_conv_desc,
                   rnn_quant_desc, rnn_scan_desc, rnn_scores_desc)

_DTYPES = {torch.float32: RNN_DTYPE_F32, torch.bfloat16: RNN_DTYPE_BF16,
           torch.float16: RNN_DTYPE_F16}

# Descriptors (with the workspace they need) by the shapes, strides and types
# of a call: a loop of equal calls is checked and described once.
_known: dict = {}


def _remember(key, value):
    if len(_known) >= 4096:
        _known.clear()
    _known[key] = value
    return value


def _no_gradient(**tensors):
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} requires a gradient, and this operator has none: call it under "
                                 "torch.no_grad(), or pass a detached tensor")


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_ENTRIES = ("rnn_conv_run", "rnn_scan_workspace_size", "rnn_scan_run", "rnn_quantize_rows",
            "rnn_quant_workspace_size", "rnn_quant_project", "rnn_scores_workspace_size",
            "rnn_token_scores")
_bound = None


def _bind():
    """The compiled module, with the entry points of the loaded library."""
    global _bound
    lib = _lib.load()
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("recurrent_nn_amd/_binding.so is missing: build it with "
                           "`python recurrent_nn_amd/build.py` (or __graft_entry__.build())") from e
    _binding.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES])
    _bound = _binding
    return _bound


def _done(r, where):
    """The outputs of a compiled call; RNNError for a status."""
    if type(r) is int:
        _check(r, where)
    return r


def _on(tensors, stream, call):
    """call(stream handle) with the tensors' device current; with a stream of
    the caller's, allocations inside belong to it and the tensors are marked
    as in use there."""
    device = tensors[0].device
    if stream is None and device.index == torch.cuda.current_device():
        return call(_raw_stream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return call(_raw_stream(device.index))
        with torch.cuda.stream(stream):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            return call(stream.cuda_stream)


def _expect(name, t, shape, dtype, device, dense=True):
    """A tensor of this shape, type and device; `dense` or with a contiguous
    last dimension."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if not t.is_contiguous() and (dense or (t.shape[-1] > 1 and t.stride(-1) != 1)):
        raise ValueError(f"{name} must {'be contiguous' if dense else 'have a contiguous last dimension'}")


def _data(name, t, dims):
    """A device tensor of a floating type with `dims` dimensions."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES or t.dim() != dims:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 device tensor with "
                         f"{dims} dimensions")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _lens(sequence_lens, batch, steps, device):
    """The lengths as a device int32 tensor.  Device tensors go as they are
    (the kernels bound them); host values are checked here."""
    if sequence_lens is None:
        return None
    t = sequence_lens
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        host = torch.as_tensor(t)
        if host.shape != (batch,) or host.is_floating_point():
            raise ValueError(f"sequence_lens must be {batch} integers")
        if batch and (int(host.min()) < 0 or int(host.max()) > steps):
            raise ValueError(f"sequence_lens outside [0, {steps}]")
        return host.to(device=device, dtype=torch.int32)
    _expect("sequence_lens", t, (batch,), torch.int32, device)
    return t


def _workspace(fn, desc):
    n = ctypes.c_size_t()
    _check(fn(ctypes.addressof(desc), ctypes.byref(n)), fn.__name__)
    return n.value


def causal_conv(x, weight, bias=None, silu: bool = False, state=None, sequence_lens=None, out=None,
                state_out=None, stream=None):
    """Causal convolution of each channel over its last ``taps`` steps.

    x [batch, steps, dim] (last dimension contiguous, other strides free);
    weight [dim, taps] and bias [dim] float32; state [batch, taps - 1, dim],
    the inputs before the first step (None = zeros); sequence_lens [batch]
    int32 on the device, or host integers.  Returns (y, state_out): y in x's
    type, the inputs before each row's length.  One new token: steps = 1.
    ``state_out`` may be ``state``.
    """
    if stream is None and getattr(x, "is_cuda", False):
        device = _device()
        r = (_bound or _bind()).conv(x, weight, bias, silu, state, sequence_lens, out, state_out,
                                     device, _raw_stream(device))
        if r is not None:
            return _done(r, "rnn_conv_run")
    _no_gradient(x=x, weight=weight, bias=bias, state=state, out=out, state_out=state_out)
    lib = _lib.load()
    silu = bool(silu)
    key = ("conv", _sig(x), _sig(weight), _sig(bias), _sig(state), _sig(out), _sig(state_out), silu)
    known = _known.get(key)
    if known is None:
        _data("x", x, 3)
        b, t, d = x.shape
        if weight.dim() != 2:
            raise ValueError("weight must be [dim, taps]")
        k = weight.shape[1]
        if k < 1:
            raise ValueError("weight must have a tap at least")
        _expect("weight", weight, (d, k), torch.float32, x.device)
        if bias is not None:
            _expect("bias", bias, (d,), torch.float32, x.device)
        for name, s in (("state", state), ("state_out", state_out)):
            if s is not None:
                _expect(name, s, (b, k - 1, d), x.dtype, x.device)
        ys = (t * d, d)
        if out is not None:
            _expect("out", out, x.shape, x.dtype, x.device, dense=False)
            ys = out.stride()
        desc = rnn_conv_desc(b, t, d, x.stride(0), x.stride(1), ys[0], ys[1], k, silu,
                             _DTYPES[x.dtype])
        known = _remember(key, (desc, ctypes.addressof(desc), (b, t, d), (b, k - 1, d)))
    _, desc, yshape, sshape = known
    if sequence_lens is not None:
        sequence_lens = _lens(sequence_lens, yshape[0], yshape[1], x.device)

    def call(s):
        y = x.new_empty(yshape) if out is None else out
        h = x.new_empty(sshape) if state_out is None else state_out
        _check(lib.rnn_conv_run(desc, s, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state),
                                _ptr(sequence_lens), y.data_ptr(), h.data_ptr()), "rnn_conv_run")
        return y, h

    return _on((x, weight, bias, state, sequence_lens, out, state_out), stream, call)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                   state=None, sequence_lens=None, out=None, state_out=None, stream=None):
    """Selective state space scan.

    x, dt, z [batch, steps, dim]; B, C [batch, steps, states] or [batch,
    steps, groups, states], all of one type (last dimension contiguous, other
    strides free); A [dim, states], D, dt_bias [dim] and state [batch, dim,
    states] float32; sequence_lens as in :func:`causal_conv`.  Returns (y,
    state_out).  One new token: steps = 1.  ``state_out`` may be ``state``.
    """
    if stream is None and getattr(x, "is_cuda", False):
        device = _device()
        r = (_bound or _bind()).scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, sequence_lens,
                                     out, state_out, device, _raw_stream(device))
        if r is not None:
            return _done(r, "rnn_scan_run")
    _no_gradient(x=x, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, state=state, out=out,
                 state_out=state_out)
    lib = _lib.load()
    dt_softplus = bool(dt_softplus)
    key = ("scan", _sig(x), _sig(dt), _sig(A), _sig(B), _sig(C), _sig(D), _sig(z), _sig(dt_bias),
           _sig(state), _sig(out), _sig(state_out), dt_softplus)
    known = _known.get(key)
    if known is None:
        _data("x", x, 3)
        b, t, d = x.shape
        if B.dim() not in (3, 4):
            raise ValueError("B must be [batch, steps, states] or [batch, steps, groups, states]")
        n, g = B.shape[-1], (B.shape[2] if B.dim() == 4 else 1)
        for name, v, shape in (("dt", dt, x.shape), ("z", z, x.shape), ("out", out, x.shape),
                               ("B", B, (b, t, g, n) if B.dim() == 4 else (b, t, n)),
                               ("C", C, B.shape)):
            if v is not None:
                _expect(name, v, shape, x.dtype, x.device, dense=False)
        for name, v, shape in (("A", A, (d, n)), ("D", D, (d,)), ("dt_bias", dt_bias, (d,)),
                               ("state", state, (b, d, n)), ("state_out", state_out, (b, d, n))):
            if v is not None:
                _expect(name, v, shape, torch.float32, x.device)
        ys = (t * d, d) if out is None else out.stride()
        zs = (0, 0) if z is None else z.stride()
        bs = B.stride() if B.dim() == 4 else (B.stride(0), B.stride(1), 0)
        cs = C.stride() if C.dim() == 4 else (C.stride(0), C.stride(1), 0)
        desc = rnn_scan_desc(b, t, d, n, g, x.stride(0), x.stride(1), dt.stride(0), dt.stride(1),
                             zs[0], zs[1], ys[0], ys[1], bs[0], bs[1], bs[2], cs[0], cs[1], cs[2],
                             _DTYPES[x.dtype], dt_softplus)
        size = _workspace(lib.rnn_scan_workspace_size, desc)
        known = _remember(key, (desc, ctypes.addressof(desc), size, (b, t, d), (b, d, n)))
    _, desc, size, yshape, sshape = known
    if sequence_lens is not None:
        sequence_lens = _lens(sequence_lens, yshape[0], yshape[1], x.device)

    def call(s):
        y = x.new_empty(yshape) if out is None else out
        h = A.new_empty(sshape) if state_out is None else state_out
        ws = A.new_empty((size + 3) // 4) if size else None
        _check(lib.rnn_scan_run(desc, s, _ptr(ws), size, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
                                B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias),
                                _ptr(state), _ptr(sequence_lens), y.data_ptr(), h.data_ptr()),
               "rnn_scan_run")
        return y, h

    return _on((x, dt, A, B, C, D, z, dt_bias, state, sequence_lens, out, state_out), stream, call)


class QuantRows(NamedTuple):
    """Rows in 8 bits: q int8 [rows, cols] (row pitch a multiple of 128
    bytes, zeros past cols) and scale float32 [rows]; q * scale is the row."""
    q: torch.Tensor
    scale: torch.Tensor


def quantize_rows(x, stream=None) -> QuantRows:
    """The rows of x [rows, cols] in 8 bits with one scale each (weights: a row
    is an output channel; activations: a row is a token)."""
    if stream is None and getattr(x, "is_cuda", False):
        device = _device()
        r = (_bound or _bind()).quantize(x, device, _raw_stream(device))
        if r is not None:
            return QuantRows._make(_done(r, "rnn_quantize_rows"))
    _no_gradient(x=x)
    lib = _lib.load()
    _data("x", x, 2)
    rows, cols = x.shape
    pitch = (cols + 127) // 128 * 128

    def call(s):
        q = x.new_empty((rows, pitch), dtype=torch.int8)
        scale = x.new_empty((rows,), dtype=torch.float32)
        _check(lib.rnn_quantize_rows(s, rows, cols, _DTYPES[x.dtype], x.data_ptr(), x.stride(0),
                                     q.data_ptr(), pitch, scale.data_ptr()), "rnn_quantize_rows")
        return QuantRows(q if pitch == cols else q[:, :cols], scale)

    return _on((x,), stream, call)


def _eight_bit(name, t, device):
    if t.dtype != torch.int8 or t.dim() != 2 or t.device != device:
        raise ValueError(f"{name} must be a two-dimensional int8 tensor on {device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")


def _readable(name, t):
    """The kernels read whole 16-byte pieces of 8-bit rows, also the last row's.
    (A pitch of as many columns is a multiple of 16, or refused as it is.)"""
    (rows, cols), pitch = t.shape, t.stride(0)
    if rows > 0 and pitch != cols and \
            t.untyped_storage().nbytes() < t.storage_offset() + (rows - 1) * pitch + (cols + 15) // 16 * 16:
        raise ValueError(f"{name}: its last row must be readable up to a multiple of 16 columns "
                         "(as within a row pitch of 16 bytes)")


def quant_project(x, w, w_scale, bias=None, x_scale=None, out_dtype: Optional[torch.dtype] = None,
                  out=None, stream=None):
    """y [rows, outs] = x [rows, cols] . w [outs, cols]^T in 8-bit integers.

    w int8 with rows at multiples of 16 bytes and w_scale [outs] float32, as
    :func:`quantize_rows` gives them; x float32, bfloat16 or float16 (rounded
    to 8 bits inside, one scale for each row), or int8 rows at multiples of 16
    bytes with x_scale [rows] float32.  8-bit rows may be columns of wider ones,
    whatever those hold.  bias [outs] float32.  y is in ``out_dtype`` (default:
    x's type, float32 for int8 rows).
    """
    if stream is None and getattr(x, "is_cuda", False):
        device = _device()
        r = (_bound or _bind()).project(x, w, w_scale, bias, x_scale, out_dtype, out, device,
                                        _raw_stream(device))
        if r is not None:
            return _done(r, "rnn_quant_project")[0]
    _no_gradient(x=x, w_scale=w_scale, bias=bias, x_scale=x_scale, out=out)
    lib = _lib.load()
    key = ("project", _sig(x), _sig(w), _sig(w_scale), _sig(bias), _sig(x_scale), out_dtype, _sig(out))
    known = _known.get(key)
    if known is None:
        eight = x.dtype == torch.int8
        if eight:
            _eight_bit("x", x, x.device)
            if not x.is_cuda or x_scale is None:
                raise ValueError("int8 rows must be on the device and come with x_scale")
            _expect("x_scale", x_scale, (x.shape[0],), torch.float32, x.device)
        else:
            _data("x", x, 2)
            if x_scale is not None:
                raise ValueError("x_scale goes with int8 rows")
        _eight_bit("w", w, x.device)
        rows, cols = x.shape
        outs = w.shape[0]
        if w.shape[1] != cols:
            raise ValueError(f"w must be [outs, {cols}]")
        _expect("w_scale", w_scale, (outs,), torch.float32, x.device)
        if bias is not None:
            _expect("bias", bias, (outs,), torch.float32, x.device)
        kind = out_dtype or (out.dtype if out is not None else torch.float32 if eight else x.dtype)
        if kind not in _DTYPES:
            raise ValueError("out_dtype must be float32, bfloat16 or float16")
        if out is not None:
            _expect("out", out, (rows, outs), kind, x.device, dense=False)
        desc = rnn_quant_desc(rows, cols, outs, x.stride(0), w.stride(0),
                              outs if out is None else out.stride(0),
                              RNN_DTYPE_I8 if eight else _DTYPES[x.dtype], _DTYPES[kind])
        size = _workspace(lib.rnn_quant_workspace_size, desc)
        known = _remember(key, (desc, ctypes.addressof(desc), size, (rows, outs), kind))
    _, desc, size, yshape, kind = known
    _readable("w", w)
    if x_scale is not None:
        _readable("x", x)

    def call(s):
        y = w_scale.new_empty(yshape, dtype=kind) if out is None else out
        ws = w_scale.new_empty((size + 3) // 4) if size else None
        _check(lib.rnn_quant_project(desc, s, _ptr(ws), size, x.data_ptr(), _ptr(x_scale),
                                     w.data_ptr(), w_scale.data_ptr(), _ptr(bias), y.data_ptr()),
               "rnn_quant_project")
        return y

    return _on((x, w, w_scale, bias, x_scale, out), stream, call)


class TokenScores(NamedTuple):
    """What rows of logits say of their tokens (see :func:`token_scores`)."""
    logprob: Optional[torch.Tensor]       # [rows] log probability of the token
    entropy: torch.Tensor                 # [rows] entropy of the distribution, in nats
    rank: Optional[torch.Tensor]          # [rows] entries before the token (int32)
    top_logprobs: torch.Tensor            # [rows, top] the most likely entries' log probabilities
    top_ids: torch.Tensor                 # [rows, top] and their indices (int32)


def token_scores(logits, tokens=None, top: int = 0, stream=None) -> TokenScores:
    """Log probability and rank of given tokens, entropy, and the ``top`` most
    likely entries (equal ones in the order of their index) of each row of
    logits [rows, vocab]; tokens [rows] int32 or int64, or None."""
    if stream is None and getattr(logits, "is_cuda", False):
        device = _device()
        r = (_bound or _bind()).scores(logits, tokens, top, device, _raw_stream(device))
        if r is not None:
            return TokenScores._make(_done(r, "rnn_token_scores"))
    _no_gradient(logits=logits)
    lib = _lib.load()
    key = ("scores", _sig(logits), _sig(tokens), top)
    known = _known.get(key)
    if known is None:
        _data("logits", logits, 2)
        rows, vocab = logits.shape
        if tokens is not None and tokens.dtype not in (torch.int32, torch.int64):
            raise ValueError("tokens must be int32 or int64")
        if tokens is not None:
            _expect("tokens", tokens, (rows,), tokens.dtype, logits.device)
        desc = rnn_scores_desc(rows, vocab, logits.stride(0), _DTYPES[logits.dtype],
                               4 if tokens is not None and tokens.dtype == torch.int32 else 8, top)
        size = _workspace(lib.rnn_scores_workspace_size, desc)
        known = _remember(key, (desc, ctypes.addressof(desc), size, rows))
    _, desc, size, rows = known

    def call(s):
        ws = logits.new_empty((size + 3) // 4, dtype=torch.float32) if size else None
        lp, en = logits.new_empty((2, rows), dtype=torch.float32).unbind(0)
        tl = logits.new_empty((rows, top), dtype=torch.float32)
        ti = logits.new_empty((rows, top), dtype=torch.int32)
        rk = None
        if tokens is None:
            lp = None
        else:
            rk = ti.new_empty(rows)
        _check(lib.rnn_token_scores(desc, s, _ptr(ws), size, logits.data_ptr(), _ptr(tokens),
                                    _ptr(lp), en.data_ptr(), _ptr(rk), tl.data_ptr(),
                                    ti.data_ptr()), "rnn_token_scores")
        return TokenScores(lp, en, rk, tl, ti)

    return _on((logits, tokens), stream, call)
