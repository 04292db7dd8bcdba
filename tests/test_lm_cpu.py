"""The language-model operators without a GPU: descriptors laid out as the
header says, every refusal raised before anything touches a device, the
binding's own checks, and the plain definitions that the GPU tests use pinned
to independent ones."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from recurrent_nn_amd import _lib
from tests import lm_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # a 256-aligned address that is never dereferenced
OK, INVALID, UNSUPPORTED = ra.RNN_OK, ra.RNN_ERR_INVALID_INPUT, ra.RNN_ERR_UNSUPPORTED


def test_descriptors_match_the_header():
    names = ["rnn_conv_desc", "rnn_scan_desc", "rnn_quant_desc", "rnn_scores_desc"]
    lines = []
    for n in names:
        lines.append(f'printf("{n} size %zu\\n", sizeof({n}));')
        for f, _ in getattr(_lib, n)._fields_:
            lines.append(f'printf("{n} {f} %zu\\n", offsetof({n}, {f}));')
    for c in ("RNN_CONV_MAX_TAPS", "RNN_SCAN_MAX_STATES", "RNN_QUANT_MAX_COLS", "RNN_SCORES_MAX_TOP",
              "RNN_DTYPE_F32", "RNN_DTYPE_BF16", "RNN_DTYPE_F16", "RNN_DTYPE_I8"):
        lines.append(f'printf("const {c} %zu\\n", (size_t){c});')
    src = '#include <stdio.h>\n#include <stddef.h>\n' \
          f'#include "{ROOT}/include/recurrent_nn_amd.h"\nint main(){{{"".join(lines)}return 0;}}'
    os.makedirs(os.path.join(ROOT, "_build"), exist_ok=True)
    c, exe = (os.path.join(ROOT, "_build", n) for n in ("lm_abi.c", "lm_abi"))
    with open(c, "w") as f:
        f.write(src)
    subprocess.run(["gcc", "-o", exe, c], check=True)
    for line in subprocess.run([exe], capture_output=True, text=True).stdout.splitlines():
        what, field, value = line.split()
        if what == "const":
            assert getattr(_lib, field) == int(value)
        elif field == "size":
            assert ctypes.sizeof(getattr(_lib, what)) == int(value)
        else:
            assert getattr(getattr(_lib, what), field).offset == int(value), line


def conv(call=None, **kw):
    f = dict(batch=2, steps=5, dim=8, x_batch_stride=40, x_step_stride=8, y_batch_stride=40,
             y_step_stride=8, taps=4, silu=0, dtype=_lib.RNN_DTYPE_BF16)
    f.update(kw)
    p = dict(x=FAKE, weight=FAKE, bias=0, state_in=0, lens=0, y=2 * FAKE, state_out=0)
    p.update(call or {})
    d = _lib.rnn_conv_desc(**f)
    return _lib.load().rnn_conv_run(ctypes.addressof(d), 0, *p.values())


def test_conv_refusals():
    for bad in (dict(batch=-1), dict(steps=-1), dict(dim=-1), dict(taps=0), dict(taps=9),
                dict(dtype=3), dict(dtype=7), dict(x_step_stride=-8), dict(y_step_stride=4),
                dict(y_batch_stride=24), dict(x_batch_stride=1 << 60), dict(batch=1 << 50)):
        assert conv(**bad) == INVALID, bad
        assert ra.rnn_last_error().startswith("rnn_conv_run: ")
    for bad in (dict(x=0), dict(weight=0), dict(y=0), dict(x=FAKE + 1), dict(weight=FAKE + 2),
                dict(bias=FAKE + 1), dict(state_in=FAKE + 1), dict(lens=FAKE + 2),
                dict(state_out=FAKE + 1), dict(y=FAKE), dict(state_in=2 * FAKE),
                dict(state_out=FAKE)):
        assert conv(bad) == INVALID, bad
    assert _lib.load().rnn_conv_run(0, 0, FAKE, FAKE, 0, 0, 0, FAKE, 0) == INVALID
    # nothing to do: accepted without tensors
    for empty in (dict(batch=0), dict(dim=0), dict(steps=0)):
        assert conv(dict(x=0, weight=0, y=0), **empty) == OK, empty


def scan(call=None, ws=(0, 0), **kw):
    f = dict(batch=2, steps=5, dim=8, states=4, groups=2, x_batch_stride=40, x_step_stride=8,
             dt_batch_stride=40, dt_step_stride=8, z_batch_stride=40, z_step_stride=8,
             y_batch_stride=40, y_step_stride=8, B_batch_stride=40, B_step_stride=8,
             B_group_stride=4, C_batch_stride=40, C_step_stride=8, C_group_stride=4,
             dtype=_lib.RNN_DTYPE_F32, dt_softplus=1)
    f.update(kw)
    p = dict(x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, D=0, z=0, dt_bias=0, state_in=0, lens=0,
             y=2 * FAKE, state_out=0)
    p.update(call or {})
    d = _lib.rnn_scan_desc(**f)
    return _lib.load().rnn_scan_run(ctypes.addressof(d), 0, *ws, *p.values())


def test_scan_refusals():
    for bad in (dict(batch=-1), dict(steps=-2), dict(dim=-8), dict(states=0), dict(states=65),
                dict(groups=0), dict(groups=3), dict(dtype=3), dict(x_step_stride=-1),
                dict(dt_batch_stride=-1), dict(B_step_stride=-1), dict(C_batch_stride=-1),
                dict(B_group_stride=-1), dict(C_group_stride=-1), dict(y_step_stride=7),
                dict(y_batch_stride=39), dict(batch=1 << 30, steps=1 << 30)):
        assert scan(**bad) == INVALID, bad
    assert scan(dict(z=FAKE), z_step_stride=-1) == INVALID
    for bad in (dict(x=0), dict(dt=0), dict(A=0), dict(B=0), dict(C=0), dict(y=0),
                dict(x=FAKE + 2), dict(dt=FAKE + 1), dict(A=FAKE + 1), dict(B=FAKE + 2),
                dict(C=FAKE + 2), dict(D=FAKE + 1), dict(z=FAKE + 2), dict(dt_bias=FAKE + 1),
                dict(state_in=FAKE + 2), dict(lens=FAKE + 1), dict(state_out=FAKE + 2),
                dict(y=FAKE), dict(z=2 * FAKE), dict(state_in=2 * FAKE), dict(state_out=2 * FAKE)):
        assert scan(bad) == INVALID, bad
    assert _lib.load().rnn_scan_run(0, 0, 0, 0, *[FAKE] * 12) == INVALID
    for empty in (dict(batch=0), dict(dim=0), dict(steps=0)):
        assert scan(dict(x=0, dt=0, A=0, B=0, C=0, y=0), **empty) == OK, empty


def test_scan_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    d = _lib.rnn_scan_desc(batch=1, steps=100000, dim=64, states=16, groups=1, dtype=1)
    assert lib.rnn_scan_workspace_size(ctypes.addressof(d), ctypes.byref(n)) == OK
    assert lib.rnn_scan_workspace_size(ctypes.addressof(d), None) == INVALID
    if n.value:         # a workspace that is missing, too small or misaligned
        big = dict(batch=1, steps=100000, dim=64, states=16, groups=1)
        for ws in ((0, 0), (FAKE, n.value - 1), (FAKE + 64, n.value)):
            assert scan(ws=ws, **big, x_step_stride=64, dt_step_stride=64, z_step_stride=64,
                        y_step_stride=64, B_step_stride=16, C_step_stride=16) == INVALID


def test_quantize_refusals():
    run = _lib.load().rnn_quantize_rows
    good = dict(stream=0, rows=3, cols=40, dtype=1, x=FAKE, x_stride=40, q=2 * FAKE, q_stride=48,
                scale=FAKE)
    for bad in (dict(rows=-1), dict(cols=-1), dict(dtype=3), dict(dtype=-1), dict(x_stride=-1),
                dict(q_stride=32), dict(q_stride=56), dict(x=0), dict(q=0), dict(scale=0),
                dict(x=FAKE + 1), dict(q=FAKE + 8), dict(scale=FAKE + 2), dict(q=FAKE)):
        assert run(*{**good, **bad}.values()) == INVALID, bad
    assert run(*{**good, "rows": 1 << 31}.values()) == UNSUPPORTED
    assert run(*{**good, "rows": 0, "x": 0, "q": 0, "scale": 0}.values()) == OK


def project(call=None, ws=(FAKE, 1 << 30), **kw):
    f = dict(rows=3, cols=40, outs=5, x_stride=40, w_stride=48, y_stride=5, x_dtype=1, y_dtype=1)
    f.update(kw)
    p = dict(x=FAKE, x_scale=0, w=FAKE, w_scale=FAKE, bias=0, y=2 * FAKE)
    p.update(call or {})
    d = _lib.rnn_quant_desc(**f)
    return _lib.load().rnn_quant_project(ctypes.addressof(d), 0, *ws, *p.values())


def test_project_refusals():
    for bad in (dict(rows=-1), dict(cols=-1), dict(outs=-1), dict(x_stride=-1), dict(w_stride=32),
                dict(w_stride=56), dict(y_stride=4), dict(x_dtype=4), dict(y_dtype=3)):
        assert project(**bad) == INVALID, bad
    for bad in (dict(cols=131072, w_stride=131072, x_stride=131072), dict(rows=1 << 31),
                dict(outs=1 << 31, y_stride=1 << 31)):
        assert project(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=0), dict(w=0), dict(w_scale=0), dict(y=0), dict(x=FAKE + 1),
                dict(w=FAKE + 8), dict(w_scale=FAKE + 1), dict(bias=FAKE + 2), dict(y=FAKE + 1),
                dict(x_scale=FAKE), dict(y=FAKE)):
        assert project(bad) == INVALID, bad
    eight = dict(x_dtype=3, x_stride=48)
    assert project(**eight) == INVALID                                      # no x_scale
    assert project(dict(x_scale=FAKE), x_dtype=3, x_stride=40) == INVALID    # pitch not of 16 bytes
    assert project(dict(x_scale=FAKE, x=FAKE + 2), **eight) == INVALID
    assert project(dict(x=0, w=0, w_scale=0, y=0), rows=0) == OK
    assert project(dict(x=0, w=0, w_scale=0, y=0), outs=0) == OK
    n = ctypes.c_size_t()
    d = _lib.rnn_quant_desc(rows=3000, cols=400, outs=500, x_stride=400, w_stride=400, y_stride=500,
                            x_dtype=1, y_dtype=1)
    assert _lib.load().rnn_quant_workspace_size(ctypes.addressof(d), ctypes.byref(n)) == OK
    assert n.value >= 3000 * 400
    big = dict(rows=3000, cols=400, outs=500, x_stride=400, w_stride=400, y_stride=500)
    for ws in ((0, n.value), (FAKE, n.value - 1), (FAKE + 128, n.value)):
        assert project(ws=ws, **big) == INVALID, ws


def scores(call=None, ws=(FAKE, 1 << 30), **kw):
    f = dict(rows=3, vocab=40, logits_stride=40, dtype=1, token_bytes=8, top=2)
    f.update(kw)
    p = dict(logits=FAKE, tokens=FAKE, logprob=FAKE, entropy=FAKE, rank=FAKE, tl=FAKE, ti=FAKE)
    p.update(call or {})
    d = _lib.rnn_scores_desc(**f)
    return _lib.load().rnn_token_scores(ctypes.addressof(d), 0, *ws, *p.values())


def test_scores_refusals():
    for bad in (dict(rows=-1), dict(vocab=0), dict(logits_stride=-1), dict(dtype=3),
                dict(token_bytes=2), dict(top=-1), dict(top=65)):
        assert scores(**bad) == INVALID, bad
    assert scores(rows=1 << 31) == UNSUPPORTED
    assert scores(vocab=(1 << 31) - 1) == UNSUPPORTED
    for bad in (dict(logits=0), dict(tokens=0), dict(logits=FAKE + 1), dict(tokens=FAKE + 4),
                dict(logprob=FAKE + 1), dict(entropy=FAKE + 1), dict(rank=FAKE + 1),
                dict(tl=FAKE + 1), dict(ti=FAKE + 1)):
        assert scores(bad) == INVALID, bad
    assert scores({k: 0 for k in ("logits", "tokens", "logprob", "entropy", "rank", "tl", "ti")},
                  rows=0) == OK


def test_binding_refuses_tensors_of_the_wrong_kind():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ra.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="device tensor"):
        ra.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4))
    with pytest.raises(ValueError, match="device tensor"):
        ra.quantize_rows(x[0])
    with pytest.raises(ValueError, match="device tensor"):
        ra.quant_project(x[0], torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="device tensor"):
        ra.token_scores(x[0])
    from recurrent_nn_amd import lm
    for bad in ([1, 2], [1, 2, 9], [1, -1, 2], [1.0, 2.0, 3.0]):
        with pytest.raises(ValueError, match="sequence_lens"):
            lm._lens(bad, 3, 8, torch.device("cpu"))
    assert lm._lens([1, 8, 0], 3, 8, torch.device("cpu")).dtype == torch.int32
    w = torch.zeros(4 * 16 - 8, dtype=torch.int8).as_strided((4, 8), (16, 1))
    with pytest.raises(ValueError, match="row pitch"):
        lm._readable("w", w)
    with pytest.raises(AttributeError):
        ra.no_such_operator


# ---------------------------------------------------------------------------
# The plain definitions against independent ones
# ---------------------------------------------------------------------------

def test_reference_conv_is_a_padded_convolution():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 9, 6, generator=g)
    w, b = torch.randn(6, 4, generator=g), torch.randn(6, generator=g)
    y, _, win = lm_ref.conv(x, w, b, True, None, None)
    ref = torch.nn.functional.conv1d(x.double().transpose(1, 2), w.double()[:, None], b.double(),
                                     padding=3, groups=6)[:, :, :9].transpose(1, 2)
    assert np.allclose(y, torch.nn.functional.silu(ref).numpy(), atol=1e-12)
    # a prompt in two parts is the prompt in one
    y1, _, w1 = lm_ref.conv(x[:, :2], w, b, True, None, None)
    y2, _, w2 = lm_ref.conv(x[:, 2:], w, b, True, torch.from_numpy(w1).float(), None)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(w2, win)


def test_reference_scan_closed_forms():
    # one state, constant step and coefficients: h is a geometric sum
    t, A, s = 7, -0.5, 0.3
    one = torch.ones(1, t, 1)
    y, _, h, _ = lm_ref.scan(one, one * s, torch.full((1, 1), A), one, one * 2, torch.full((1,), 3.0),
                             None, None, False, None, None)
    a = np.exp(np.float64(np.float32(s)) * A)
    want = np.float64(np.float32(s)) * (1 - a ** np.arange(1, t + 1)) / (1 - a)
    assert np.allclose(y[0, :, 0], 2 * want + 3, rtol=1e-12) and np.isclose(h[0, 0, 0], want[-1])
    # no step size leaves the state as it is
    g = torch.Generator().manual_seed(5)
    h0 = torch.randn(2, 4, 3, generator=g)
    x, B = torch.randn(2, 5, 4, generator=g), torch.randn(2, 5, 3, generator=g)
    _, _, h, _ = lm_ref.scan(x, x * 0, -torch.rand(4, 3, generator=g), B, B, None, None, None, False,
                             h0, None)
    assert np.array_equal(h, h0.double().numpy())


def test_reference_scores():
    x = torch.tensor([[1.0, 3.0, 3.0, -float("inf"), 2.0]])
    s = lm_ref.scores(x, torch.tensor([2]), 3)
    p = torch.log_softmax(x.double(), 1)[0]
    assert s["top_ids"].tolist() == [[1, 2, 4]] and s["rank"][0] == 1
    assert np.isclose(s["logprob"][0], p[2]) and np.isclose(
        s["entropy"][0], torch.distributions.Categorical(logits=x.double()).entropy()[0])
    x[0, 3] = float("nan")
    s = lm_ref.scores(x, torch.tensor([9]), 2)
    assert s["top_ids"].tolist() == [[3, 1]] and s["rank"][0] == -1 and np.isnan(s["entropy"][0])


def test_reference_quantize():
    x = torch.tensor([[1.0, -2.0, 0.5], [0, 0, 0], [1, float("inf"), 0], [float("nan"), 1, 2]])
    q, s = lm_ref.quantize(x)
    assert q[0].tolist() == [64, -127, 32] and s[0] == np.float32(2) / np.float32(127)
    assert not q[1:].any() and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3])


def test_column_slices_of_8_bit_rows_are_readable():
    from recurrent_nn_amd import lm
    w = torch.zeros(64, 2048, dtype=torch.int8)
    for lo, hi in ((0, 2048), (1024, 2048), (2032, 2048), (2032, 2047), (16, 17), (0, 1000)):
        lm._readable("w", w[:, lo:hi])
    lm._readable("w", w[:0, 16:])
    dense = torch.zeros(4 * 16, dtype=torch.int8)
    lm._readable("w", dense.as_strided((4, 8), (16, 1)))
    for cut in (1, 5, 8):                   # the last row's piece of 16 bytes is cut off
        with pytest.raises(ValueError, match="row pitch"):
            lm._readable("w", dense[:-cut].clone().as_strided((4, 8), (16, 1), 0))
    with pytest.raises(ValueError, match="w:"):
        lm._readable("w", w.flatten()[:-9].clone().as_strided((64, 1999), (2048, 1), 40))


def test_launches_of_too_many_threads_are_refused():
    # (each of these is one more than a grid of 32 bits of threads takes, or a little more)
    ws = (FAKE, 1 << 62)
    one = dict(x_batch_stride=1, x_step_stride=1, y_batch_stride=1, y_step_stride=1)
    assert conv(batch=1 << 32, steps=1, dim=1, **one) == UNSUPPORTED
    assert ra.rnn_last_error() == "rnn_conv_run: more work than one launch takes"
    wide = dict(groups=1, states=16, B_batch_stride=0, B_step_stride=0, C_batch_stride=0, C_step_stride=0,
                x_batch_stride=0, x_step_stride=0, dt_batch_stride=0, dt_step_stride=0)
    assert scan(ws=ws, batch=1 << 20, steps=1, dim=1024, y_batch_stride=1024, y_step_stride=1024,
                **wide) == UNSUPPORTED
    assert scan(ws=ws, batch=1 << 20, steps=65, dim=128, y_batch_stride=65 * 128, y_step_stride=128,
                **wide) == UNSUPPORTED
    assert scan(dict(state_out=FAKE), ws=ws, batch=1 << 20, steps=0, dim=512, **wide) == UNSUPPORTED
    run = _lib.load().rnn_quantize_rows
    for rows, cols in ((1 << 24, 2049), (1 << 24, 32768), (1 << 22, 32769), (1 << 26, 2048), (1 << 28, 500),
                       (1 << 30, 100)):
        pitch = (cols + 15) // 16 * 16
        assert run(0, rows, cols, 1, FAKE, 0, 2 * FAKE, pitch, FAKE) == UNSUPPORTED, (rows, cols)
    eight = dict(x_scale=FAKE)
    for call, f in (({}, dict(rows=1, cols=16, outs=1 << 28, x_stride=16)),
                    ({}, dict(rows=16, cols=1000, outs=1 << 28, x_stride=1008)),
                    ({}, dict(rows=1 << 20, cols=16, outs=1 << 20, x_stride=16)),
                    (eight, dict(rows=1 << 20, cols=16, outs=1 << 20, x_stride=16, x_dtype=3))):
        assert project(call, ws=ws, w_stride=1008, y_stride=f["outs"], **f) == UNSUPPORTED, f
    for rows, vocab in ((1 << 26, 8), (1 << 24, 4096)):
        assert scores(ws=ws, rows=rows, vocab=vocab, logits_stride=0) == UNSUPPORTED
