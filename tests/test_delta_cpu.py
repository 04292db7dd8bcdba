"""The delta-rule operators and those of decoding with several beams without a
GPU: descriptors laid out as the header says, every refusal raised before
anything touches a device, the binding's own checks, and the plain definitions
that the GPU tests use pinned to independent ones."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from recurrent_nn_amd import _lib, delta, lm
from tests import delta_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # a 256-aligned address that is never dereferenced
OK, INVALID, UNSUPPORTED = ra.RNN_OK, ra.RNN_ERR_INVALID_INPUT, ra.RNN_ERR_UNSUPPORTED


def test_descriptors_match_the_header():
    lines = []
    for n in ("rnn_delta_desc", "rnn_norm_desc", "rnn_beam_desc", "rnn_reorder_item"):
        lines.append(f'printf("{n} size %zu\\n", sizeof({n}));')
        for f, _ in getattr(_lib, n)._fields_:
            lines.append(f'printf("{n} {f} %zu\\n", offsetof({n}, {f.rstrip("_")}));')
    for c in ("RNN_DELTA_MAX_KEY_DIM", "RNN_BEAM_MAX", "RNN_REORDER_MAX_BEAMS"):
        lines.append(f'printf("const {c} %zu\\n", (size_t){c});')
    src = '#include <stdio.h>\n#include <stddef.h>\n' \
          f'#include "{ROOT}/include/recurrent_nn_amd.h"\nint main(){{{"".join(lines)}return 0;}}'
    os.makedirs(os.path.join(ROOT, "_build"), exist_ok=True)
    c, exe = (os.path.join(ROOT, "_build", n) for n in ("delta_abi.c", "delta_abi"))
    with open(c, "w") as f:
        f.write(src)
    subprocess.run(["gcc", "-o", exe, c], check=True)
    out = subprocess.run([exe], capture_output=True, text=True).stdout.splitlines()
    assert len(out) == len(lines)
    for line in out:
        what, field, value = line.split()
        if what == "const":
            assert getattr(_lib, field) == int(value)
        elif field == "size":
            assert ctypes.sizeof(getattr(_lib, what)) == int(value)
        else:
            assert getattr(getattr(_lib, what), field).offset == int(value), line


def run_delta(call=None, ws=(0, 0), **kw):
    f = dict(batch=2, steps=3, key_heads=2, heads=4, key_dim=8, value_dim=16,
             q_batch_stride=48, q_step_stride=16, q_head_stride=8, k_batch_stride=48, k_step_stride=16,
             k_head_stride=8, v_batch_stride=192, v_step_stride=64, v_head_stride=16, o_batch_stride=192,
             o_step_stride=64, o_head_stride=16, beta_batch_stride=12, beta_step_stride=4,
             g_batch_stride=12, g_step_stride=4, dtype=1, gate_dtype=0, normalize=0, beta_sigmoid=0, scale=0.5)
    f.update(kw)
    p = dict(q=FAKE, k=FAKE, v=FAKE, beta=FAKE, g=0, A=0, dt_bias=0, state_in=0, lens=0, o=2 * FAKE, state_out=0)
    p.update(call or {})
    d = _lib.rnn_delta_desc(**f)
    return _lib.load().rnn_delta_run(ctypes.addressof(d), 0, *ws, *p.values())


def test_delta_refusals():
    for bad in (dict(batch=-1), dict(steps=-1), dict(heads=-4), dict(value_dim=-1), dict(key_heads=0),
                dict(key_heads=3), dict(key_dim=0), dict(key_dim=257), dict(dtype=3), dict(dtype=-1),
                dict(gate_dtype=2), dict(gate_dtype=3), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(q_step_stride=-1), dict(k_head_stride=-1), dict(v_batch_stride=-1),
                dict(beta_step_stride=-1), dict(o_step_stride=63), dict(o_head_stride=15),
                dict(o_batch_stride=191), dict(o_head_stride=0), dict(batch=1 << 30, steps=1 << 30),
                dict(q_batch_stride=1 << 60)):
        assert run_delta(**bad) == INVALID, bad
        assert ra.rnn_last_error().startswith("rnn_delta_run: ")
    assert run_delta(dict(g=FAKE), g_step_stride=-1) == INVALID
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(beta=0), dict(o=0), dict(q=FAKE + 1), dict(k=FAKE + 1),
                dict(v=FAKE + 1), dict(beta=FAKE + 2), dict(g=FAKE + 2), dict(A=FAKE), dict(g=FAKE, A=FAKE + 2),
                dict(g=FAKE, dt_bias=FAKE), dict(state_in=FAKE + 2), dict(lens=FAKE + 2), dict(o=2 * FAKE + 1),
                dict(state_out=FAKE + 2), dict(o=FAKE), dict(state_in=2 * FAKE), dict(state_out=2 * FAKE),
                dict(g=2 * FAKE)):
        assert run_delta(bad) == INVALID, bad
    assert run_delta(steps=1 << 31, batch=1) == UNSUPPORTED
    assert run_delta(dict(state_out=FAKE), batch=1 << 30, steps=0) == UNSUPPORTED        # threads
    assert _lib.load().rnn_delta_run(0, 0, 0, 0, *[FAKE] * 11) == INVALID
    none = dict(q=0, k=0, v=0, beta=0, o=0)
    for empty in (dict(batch=0), dict(heads=0), dict(value_dim=0), dict(steps=0)):
        assert run_delta(none, **empty) == OK, empty


def test_delta_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    d = _lib.rnn_delta_desc(batch=1, steps=5000, key_heads=2, heads=4, key_dim=128, value_dim=128, dtype=1)
    assert lib.rnn_delta_workspace_size(ctypes.addressof(d), ctypes.byref(n)) == OK
    assert lib.rnn_delta_workspace_size(ctypes.addressof(d), None) == INVALID
    assert lib.rnn_delta_workspace_size(None, ctypes.byref(n)) == INVALID
    if n.value:         # a workspace that is missing, too small or misaligned
        big = dict(batch=1, steps=5000, key_dim=128, value_dim=128, q_step_stride=256, k_step_stride=256,
                   v_step_stride=512, o_step_stride=512, q_head_stride=128, k_head_stride=128,
                   v_head_stride=128, o_head_stride=128)
        for ws in ((0, 0), (FAKE, n.value - 1), (FAKE + 64, n.value)):
            assert run_delta(ws=ws, **big) == INVALID


def run_norm(call=None, **kw):
    f = dict(rows=3, groups=2, dim=8, x_row_stride=16, x_group_stride=8, z_row_stride=16, z_group_stride=8,
             y_row_stride=16, y_group_stride=8, weight_group_stride=0, dtype=1, gate_first=0, eps=1e-6)
    f.update(kw)
    p = dict(x=FAKE, weight=FAKE, z=0, y=2 * FAKE)
    p.update(call or {})
    d = _lib.rnn_norm_desc(**f)
    return _lib.load().rnn_gated_norm(ctypes.addressof(d), 0, *p.values())


def test_norm_refusals():
    for bad in (dict(rows=-1), dict(groups=-1), dict(dim=-1), dict(dtype=3), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x_row_stride=-1), dict(x_group_stride=-1),
                dict(y_row_stride=15), dict(y_group_stride=7), dict(gate_first=1), dict(weight_group_stride=-1)):
        assert run_norm(**bad) == INVALID, bad
        assert ra.rnn_last_error().startswith("rnn_gated_norm: ")
    assert run_norm(dict(z=FAKE), z_row_stride=-1) == INVALID
    for bad in (dict(x=0), dict(weight=0), dict(y=0), dict(x=FAKE + 1), dict(weight=FAKE + 2), dict(z=FAKE + 1),
                dict(y=FAKE + 1)):
        assert run_norm(bad) == INVALID, bad
    # in place with other strides than the input's
    assert run_norm(dict(y=FAKE), y_row_stride=32) == INVALID
    assert run_norm(dict(z=2 * FAKE), z_group_stride=0) == INVALID
    assert run_norm(dim=1 << 30, x_group_stride=1 << 30, x_row_stride=1 << 31, y_group_stride=1 << 30,
                    y_row_stride=1 << 31) == UNSUPPORTED
    assert run_norm(rows=1 << 33) == UNSUPPORTED
    for empty in (dict(rows=0), dict(groups=0), dict(dim=0)):
        assert run_norm(dict(x=0, weight=0, y=0), **empty) == OK, empty
    assert _lib.load().rnn_gated_norm(0, 0, FAKE, FAKE, 0, FAKE) == INVALID


def run_beam(call=None, ws=(FAKE, 1 << 40), **kw):
    f = dict(batch=2, beams=3, vocab=10, logits_batch_stride=30, logits_beam_stride=10, dtype=1, keep=4, eos=2)
    f.update(kw)
    p = dict(logits=FAKE, scores=FAKE, finished=0, out_scores=2 * FAKE, out_tokens=3 * FAKE, out_parents=4 * FAKE)
    p.update(call or {})
    d = _lib.rnn_beam_desc(**f)
    return _lib.load().rnn_beam_select(ctypes.addressof(d), 0, *ws, *p.values())


def test_beam_refusals():
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=65), dict(vocab=0), dict(keep=0), dict(keep=65),
                dict(dtype=3), dict(logits_batch_stride=-1), dict(logits_beam_stride=-1)):
        assert run_beam(**bad) == INVALID, bad
        assert ra.rnn_last_error().startswith("rnn_beam_select: ")
    for bad in (dict(eos=-1), dict(eos=10)):
        assert run_beam(dict(finished=FAKE), **bad) == INVALID, bad
    for bad in (dict(logits=0), dict(scores=0), dict(out_scores=0), dict(out_tokens=0), dict(out_parents=0),
                dict(logits=FAKE + 1), dict(scores=FAKE + 2), dict(out_scores=FAKE + 1), dict(out_tokens=FAKE + 2),
                dict(out_parents=FAKE + 2), dict(out_scores=FAKE), dict(out_parents=3 * FAKE)):
        assert run_beam(bad) == INVALID, bad
    assert run_beam(vocab=(1 << 31) - 65536) == UNSUPPORTED
    assert run_beam(batch=1 << 30) == UNSUPPORTED
    n, d = ctypes.c_size_t(), _lib.rnn_beam_desc(batch=2, beams=3, vocab=100000, dtype=1, keep=4)
    size = _lib.load().rnn_beam_workspace_size
    assert size(ctypes.addressof(d), ctypes.byref(n)) == OK and n.value > 0
    assert size(ctypes.addressof(d), None) == INVALID and size(None, ctypes.byref(n)) == INVALID
    for ws in ((0, 0), (FAKE, 8), (FAKE + 64, 1 << 40)):
        assert run_beam(ws=ws) == INVALID
    assert run_beam(dict(logits=0, scores=0, out_scores=0, out_tokens=0, out_parents=0), ws=(0, 0), batch=0) == OK


def run_reorder(items, batch=2, beams=3, keep=3, parents=FAKE):
    a = (_lib.rnn_reorder_item * max(1, len(items)))(*items)
    return _lib.load().rnn_reorder_states(0, batch, beams, keep, parents, ctypes.addressof(a), len(items))


def test_reorder_refusals():
    good = (FAKE, 2 * FAKE, 1, 100)
    for bad in (dict(batch=-1), dict(beams=0), dict(keep=-1), dict(parents=0), dict(parents=FAKE + 2)):
        assert run_reorder([good], **bad) == INVALID, bad
        assert ra.rnn_last_error().startswith("rnn_reorder_states: ")
    for bad in ((0, FAKE, 1, 8), (FAKE, 0, 1, 8), (FAKE, FAKE + 599, 1, 100), (FAKE + 599, FAKE, 1, 100),
                (FAKE, 2 * FAKE, -1, 8), (FAKE, 2 * FAKE, 1, -8), (FAKE, 2 * FAKE, 1 << 40, 1 << 40)):
        assert run_reorder([good, bad]) == INVALID, bad
    assert run_reorder([(FAKE, FAKE, 1, 8)], keep=2) == INVALID
    assert run_reorder([(FAKE, FAKE, 1, 8)], beams=65, keep=65) == UNSUPPORTED
    far = 1 << 45
    assert run_reorder([(far, 2 * far, 1 << 20, 1 << 20)]) == UNSUPPORTED
    # an item of a later launch that does not fit: nothing is enqueued
    assert run_reorder([(FAKE, 2 * FAKE, 1, 0)] * 40 + [(far, 2 * far, 1 << 20, 1 << 20)]) == UNSUPPORTED
    lib = _lib.load()
    assert lib.rnn_reorder_states(0, 2, 3, 3, FAKE, None, 1) == INVALID
    assert run_reorder([]) == OK and run_reorder([(0, 0, 0, 8), (0, 0, 1, 0)]) == OK
    assert run_reorder([(0, 0, 1, 8)], batch=0, parents=0) == OK


def test_reorder_items_on_each_other_are_refused():
    """Items run beside each other: a result where another item, or the choice of rows,
    is read or written would depend on which comes first.  (An item that no launch takes
    stands last, so that nothing runs; rows of 8 bytes, 48 an item, 24 the parents.)"""
    def at(i, o):
        return (FAKE + i, FAKE + o, 1, 8)

    def run(items, parents=FAKE + (1 << 20)):
        return run_reorder([*items, (1 << 45, 1 << 46, 1 << 20, 1 << 20)], parents=parents)

    for items in ([at(0, 48), at(48, 96)], [at(48, 96), at(0, 48)], [at(0, 48), at(48, 0)], [at(0, 48), at(96, 48)],
                  [at(0, 0), at(0, 0)], [at(0, 0), at(0, 48)], [at(0, 48), at(96, 144), at(200, 136)],
                  [at(0, 48), at(95, 200)], [at(0, 48), at(200, 1)],
                  [at(1000 * k, 1000 * k + 48) for k in range(50)] + [at(60000, 47)]):
        assert run(items) == INVALID, items
    for place in (48, 28, 92):
        assert run([at(0, 48)], FAKE + place) == INVALID, place
    for place in (0, 24, 96):
        assert run([at(0, 48)], FAKE + place) == UNSUPPORTED, place
    for items in ([at(0, 48), at(0, 96)], [at(0, 72), at(24, 120)], [at(0, 0), at(48, 48)], [at(0, 48), at(96, 144)],
                  [at(0, 48), (FAKE + 48, FAKE + 48, 1, 0)], [at(1000 * k, 1000 * k + 48) for k in range(50)]):
        assert run(items) == UNSUPPORTED, items



# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------

def inputs(device):
    """(call, its float inputs by name) of each operator."""
    def new(*shape):
        return torch.full(shape, 0.25, device=device)
    parents = torch.zeros(2, 2, dtype=torch.int32, device=device)
    return {
        "delta": (lambda **t: ra.gated_delta(**t),
                  dict(q=new(2, 3, 1, 8), k=new(2, 3, 1, 8), v=new(2, 3, 2, 4), beta=new(2, 3, 2), g=-new(2, 3, 2),
                       A=-new(2), dt_bias=new(2), state=new(2, 2, 8, 4))),
        "norm": (ra.gated_norm, dict(x=new(3, 2, 16), weight=new(16), z=new(3, 2, 16))),
        "beam": (ra.beam_select, dict(logits=new(2, 3, 16), scores=new(2, 3))),
        "reorder": (lambda **t: ra.reorder_states(list(t.values()), parents), {"states[0]": new(4, 3),
                                                                              "states[1]": new(4, 2, 5)}),
    }


GRADIENTS = [(op, name) for op, (_, tensors) in inputs("cpu").items() for name in tensors]


@pytest.mark.parametrize("op,name", GRADIENTS)
def test_an_input_that_requires_a_gradient_is_refused(op, name):
    call, tensors = inputs("cpu")[op]
    tensors[name].requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        call(**tensors)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):        # its place is the next thing
        call(**tensors)


@pytest.mark.gpu
@pytest.mark.parametrize("op,name", GRADIENTS)
def test_on_the_device(op, name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    call, tensors = inputs("cuda")[op]
    want = call(**tensors)
    tensors[name].requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        call(**tensors)
    with torch.no_grad():
        got = call(**tensors)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_entry_points():
    assert set(delta._ENTRIES) <= set(_lib.EXPORTED)
    compiled = delta._bind()
    with pytest.raises(TypeError):
        compiled.bind_delta(1)
    for f in (compiled.delta, compiled.norm, compiled.beam, compiled.reorder):
        with pytest.raises(TypeError):
            f(None)


def test_other_tensors_are_left_to_python():
    compiled = delta._bind()
    x, none = torch.zeros(2, 3, 2, 8), [None] * 12
    for bad in (x, None, 5, "x"):
        assert compiled.delta(bad, x, x, x, *none[:3], False, False, None, *none[:4], 0, 0) is None
        assert compiled.norm(bad, x, None, False, 1e-6, None, 0, 0) is None
        assert compiled.beam(bad, x, None, None, None, 0, 0) is None
        assert compiled.reorder([bad], bad, 0, None, 0, 0) is None
        assert compiled.reorder(bad, x, 0, None, 0, 0) is None


PROGRAM = """
import sys, warnings
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from recurrent_nn_amd import delta, lm

warnings.simplefilter("ignore")
op, kind = sys.argv[1:]
compiled = delta._bind()
lm._device, lm._raw_stream = (lambda: 0), (lambda index: 0)
none = [None] * 8
with FakeTensorMode(allow_non_fake_inputs=True):
    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    parents = new(2, 2, dtype=torch.int32)
    calls = {
        "delta": (new(5, 2, 3, 1, 8), lambda x: (x, x, new(2, 3, 2, 4), new(2, 3, 2), None, None, None, False,
                                                 False, None, None, None, new(2, 3, 2, 4), new(2, 2, 8, 4)),
                  delta.gated_delta),
        "norm": (new(5, 3, 16), lambda x: (x, new(16), None, False, 1e-6, new(3, 16)), delta.gated_norm),
        "beam": (new(5, 2, 3, 16), lambda x: (x, new(2, 3), None, None, None), delta.beam_select),
        "reorder": (new(5, 4, 3), lambda x: ([x], parents, 0, [new(4, 3)]), delta.reorder_states),
    }
    x, args, public = calls[op]
    seen = []

    def under(v):
        # the compiled call leaves it to Python, which says what is wrong
        seen.append(getattr(compiled, op)(*args(v), 0, 0))
        try:
            public(*args(v))
        except (RuntimeError, ValueError) as e:
            seen.append(e)
        return v

    if kind == "vmap":
        torch.vmap(under)(x)
    elif kind == "vjp":
        torch.func.vjp(under, x[0])
    else:
        torch.func.jvp(under, (x[0],), (x[0],))
assert seen[0] is None and isinstance(seen[1], (RuntimeError, ValueError)), seen
print("said:", seen[1])
"""


@pytest.mark.parametrize("op,kind", [("delta", "vmap"), ("norm", "vjp"), ("beam", "vmap"), ("reorder", "vmap"),
                                     ("reorder", "jvp"), ("delta", "jvp")])
def test_a_transform_is_an_error_and_no_crash(op, kind):
    r = subprocess.run([sys.executable, "-c", PROGRAM, op, kind], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0 and "said:" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])


def test_python_checks():
    """What the way without the compiled call says of tensors of the wrong kind."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    side = object()             # a stream: the compiled call is left out, and the checks come first

    with FakeTensorMode():
        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        good = dict(q=new(2, 3, 1, 8), k=new(2, 3, 1, 8), v=new(2, 3, 2, 4), beta=new(2, 3, 2), stream=side)
        for bad, what in ((dict(q=new(3, 1, 8)), "q"), (dict(q=new(2, 3, 1, 8, dtype=torch.float64)), "q"),
                          (dict(k=new(2, 3, 2, 8)), "k"), (dict(k=new(2, 3, 1, 8, dtype=torch.float16)), "k"),
                          (dict(v=new(2, 4, 2, 4)), "v"), (dict(beta=new(2, 3, 1)), "beta"),
                          (dict(beta=new(2, 3, 2, dtype=torch.bfloat16)), "beta"),
                          (dict(g=new(2, 3, 2, dtype=torch.bfloat16)), "g"), (dict(g=new(2, 3, 2), A=new(3)), "A"),
                          (dict(state=new(2, 2, 4, 8)), "state"), (dict(state_out=new(2, 2, 8, 8)[..., :4]), "state_out"),
                          (dict(out=new(2, 3, 2, 4, dtype=torch.float16)), "out"),
                          (dict(sequence_lens=[1, 2, 3]), "sequence_lens"),
                          (dict(sequence_lens=new(2, dtype=torch.int64)), "sequence_lens"),
                          (dict(q=new(2, 3, 8, 1).transpose(2, 3)[:, :, :, ::2]), "")):
            with pytest.raises(ValueError, match=what):
                ra.gated_delta(**{**good, **bad})
        good = dict(x=new(3, 2, 16), weight=new(16), stream=side)
        for bad, what in ((dict(x=new(16)), "x"), (dict(weight=new(15)), "weight"), (dict(weight=new(3, 16)), "weight"),
                          (dict(z=new(3, 2, 15)), "z"), (dict(z=new(3, 2, 16, dtype=torch.float16)), "z"),
                          (dict(out=new(3, 2, 17)), "out")):
            with pytest.raises(ValueError, match=what):
                ra.gated_norm(**{**good, **bad})
        good = dict(logits=new(2, 3, 16), scores=new(2, 3), stream=side)
        for bad, what in ((dict(logits=new(6, 16)), "logits"), (dict(scores=new(2, 4)), "scores"),
                          (dict(scores=new(2, 3, dtype=torch.float64)), "scores"),
                          (dict(finished=new(2, 3, dtype=torch.bool)), "eos"),
                          (dict(finished=new(2, 3, dtype=torch.int32), eos=1), "finished")):
            with pytest.raises(ValueError, match=what):
                ra.beam_select(**{**good, **bad})
        parents = new(2, 3, dtype=torch.int32)
        for states, more, what in (([new(5, 4)], {}, "rows"), ([new(6, 4), new(8, 4)], {}, "rows"),
                                   ([new(6, 8)[:, ::2]], {}, "contiguous"), ([new(6, 4)], dict(dim=2), "dimension"),
                                   ([new(6, 4)], dict(dim=[0, 0]), "dim"), ([new(6, 4)], dict(out=[new(6, 5)]), "out"),
                                   ([new(6, 4)], dict(out=[]), "out"), ([new(0, 4)], {}, "beam"),
                                   ([torch.empty(6, 4, device="cpu")], {}, "contiguous")):
            with pytest.raises(ValueError, match=what):
                ra.reorder_states(states, parents, stream=side, **more)
        with pytest.raises(ValueError, match="parents"):
            ra.reorder_states([new(6, 4)], new(2, 3, dtype=torch.int64), stream=side)


# ---------------------------------------------------------------------------
# The plain definitions
# ---------------------------------------------------------------------------

def test_delta_reference_by_hand():
    one = torch.ones(1, 2, 1, 1)
    o, _, S, _ = delta_ref.delta(one, one, 3 * one, torch.tensor([[[0.5], [0.5]]]), g=torch.tensor([[[0.0], [-INF]]]))
    # S = 0 + 0.5 (3 - 0) = 1.5; then forgotten, and 1.5 again
    assert np.allclose(o.ravel(), [1.5, 1.5]) and np.allclose(S.ravel(), [1.5])
    o, _, S, _ = delta_ref.delta(one, 2 * one, 3 * one, torch.ones(1, 2, 1), scale=2.0)
    # S = 2 (3 - 0) = 6; S = 6 + 2 (3 - 12) = -12
    assert np.allclose(o.ravel(), [12, -24]) and np.allclose(S.ravel(), [-12])


INF = float("inf")


def test_delta_reference_is_online_least_squares():
    """Orthonormal keys, rate 1, no decay: the state answers each key with its value."""
    gen = torch.Generator().manual_seed(1)
    k = torch.linalg.qr(torch.randn(8, 8, generator=gen, dtype=torch.float64))[0].float().view(1, 8, 1, 8)
    v = torch.randn(1, 8, 1, 5, generator=gen)
    o, err, S, S_err = delta_ref.delta(k, k, v, torch.ones(1, 8, 1), scale=1.0)
    assert np.allclose(k[0, :, 0].double().numpy() @ S[0, 0], v[0, :, 0].numpy(), atol=1e-6)
    assert np.allclose(o, v.numpy(), atol=1e-6) and (err > 0).all() and S_err.max() < 1e-3


def test_norm_reference():
    gen = torch.Generator().manual_seed(2)
    x, w, z = torch.randn(3, 2, 9, generator=gen), torch.randn(9, generator=gen), torch.randn(3, 2, 9, generator=gen)
    y, err = delta_ref.norm(x, w, None, False, 1e-5)
    want = torch.nn.functional.rms_norm(x.double(), (9,), w.double(), 1e-5)
    assert np.allclose(y, want.numpy()) and (err > 0).all()
    gate = torch.nn.functional.silu(z.double())
    assert np.allclose(delta_ref.norm(x, w, z, False, 1e-5)[0], (want * gate).numpy())
    want = torch.nn.functional.rms_norm(x.double() * gate, (9,), w.double(), 1e-5)
    assert np.allclose(delta_ref.norm(x, w, z, True, 1e-5)[0], want.numpy())


def test_beam_reference():
    x = torch.log(torch.tensor([[[0.5, 0.3, 0.2], [0.6, 0.4, 1e-30]]]))
    s, t, p = delta_ref.beam(x, torch.tensor([[0.0, -0.1]]), 4)
    assert t.tolist() == [[0, 0, 1, 1]] and p.tolist() == [[1, 0, 1, 0]]
    assert np.allclose(s, [[np.log(0.6) - 0.1, np.log(0.5), np.log(0.4) - 0.1, np.log(0.3)]], atol=1e-6)
    s, t, p = delta_ref.beam(x, torch.tensor([[0.0, -0.6]]), 7, torch.tensor([[False, True]]), 1)
    # the finished beam by itself, its other tokens at the end; no seventh
    assert t.tolist() == [[1, 0, 1, 2, 0, 2, -1]] and p.tolist() == [[1, 0, 0, 0, 1, 1, -1]]
    assert np.isneginf(s[0, 4:]).all()


def test_reorder_reference():
    x = torch.arange(12).view(2, 6)
    parents = torch.tensor([[1, 0], [1, 1], [0, 9]], dtype=torch.int32)
    assert delta_ref.reorder(x, parents, 1).tolist() == [[1, 0, 3, 3, 4, 5], [7, 6, 9, 9, 10, 11]]
