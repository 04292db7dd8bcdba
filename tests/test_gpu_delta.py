"""The gated delta rule on the GPU against its plain 64-bit definition
(tests/delta_ref.py), within bounds that count the roundings of a float32
evaluation."""
import ctypes

import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from recurrent_nn_amd import _lib
from tests import delta_ref
from tests.lm_ref import HALF_STEP, U, assert_close
from tests.test_gpu_lm import BF16, F16, F32, INF, NAN, Draw, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ra._lib.load()
    yield


def inside(t, pad, fill=NAN):
    """t as a view into a larger device tensor whose rest is `fill`; a pad of
    rows between the second-last dimension's too where there are four."""
    rows = 1 if pad and t.dim() == 4 else 0
    shape = (*t.shape[:-2], t.shape[-2] + 2 * rows, t.shape[-1] + 2 * pad)
    big = torch.full(shape, fill, dtype=t.dtype, device="cuda")
    view = big[..., rows:rows + t.shape[-2], pad:pad + t.shape[-1]]
    view.copy_(t)
    return view


def case(r, b, t, kh, h, dk, dv, dtype, gates, normalize, state, lens):
    """Keyword arguments of a call, on the host.  gates: "raw" (through A, the
    bias and the sigmoid, of dtype), "raw32" (the same in float32), "log", None."""
    x = {"q": r.normal(b, t, kh, dk), "k": r.normal(b, t, kh, dk), "v": r.normal(b, t, h, dv)}
    if not normalize:
        for n in ("q", "k"):
            x[n] = x[n] / x[n].norm(dim=-1, keepdim=True).clamp(min=1e-3)
    x = {n: v.to(dtype) for n, v in x.items()}
    raw = gates in ("raw", "raw32")
    kind = dtype if gates == "raw" else F32
    x["beta"] = (r.normal(b, t, h) if raw else r.uniform(b, t, h)).to(kind)
    x["g"] = None
    if gates:
        x["g"] = (r.normal(b, t, h) if raw else -r.uniform(b, t, h, hi=0.7) ** 2).to(kind)
    if raw:
        x["A"], x["dt_bias"] = -r.uniform(h, lo=0.1, hi=4.0), r.normal(h) - 3
    x["beta_sigmoid"], x["normalize"] = raw, normalize
    x["state"] = r.normal(b, h, dk, dv) if state else None
    x["sequence_lens"] = r.lens(b, t) if lens else None
    return x


def expected(x):
    x = dict(x)
    x["lens"] = x.pop("sequence_lens", None)
    return delta_ref.delta(**x)


def on_device(x, pad=0):
    out = {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in x.items()}
    for n in ("q", "k", "v", "beta", "g"):
        if pad and x[n] is not None:
            out[n] = inside(x[n], pad)
    if x["sequence_lens"] is not None:         # what a mask leaves out may hold anything
        for n in ("q", "k", "v", "beta", "g"):
            if x[n] is not None:
                for i, m in enumerate(x["sequence_lens"].tolist()):
                    out[n][i, m:] = NAN
    return out


CASES = [  # batch, steps, key heads, heads, key dim, value dim, dtype, gates, normalize, state, lens, pad
    (1, 1, 1, 1, 1, 1, F32, None, False, False, False, 0),
    (2, 1, 2, 4, 128, 128, BF16, "raw", True, True, False, 0),
    (3, 1, 3, 3, 96, 100, F16, "raw32", True, True, True, 8),
    (2, 1, 1, 2, 256, 33, F32, "log", False, True, False, 1),
    (3, 2, 2, 2, 64, 64, BF16, "log", False, True, True, 0),
    (2, 3, 1, 3, 17, 5, F32, "raw", True, False, False, 3),
    (1, 31, 2, 2, 32, 32, F16, "log", True, True, False, 0),
    (2, 33, 1, 1, 100, 70, BF16, None, True, False, True, 2),
    (1, 63, 1, 2, 128, 128, F32, "raw", True, True, False, 0),
    (2, 64, 2, 2, 128, 64, BF16, "raw", True, False, False, 0),
    (2, 65, 1, 2, 64, 128, F16, "raw", True, True, True, 8),
    (5, 130, 1, 1, 8, 3, F32, "log", False, True, True, 1),
    (2, 200, 2, 2, 96, 100, F16, "raw", True, True, False, 0),
    (3, 257, 1, 2, 64, 64, F32, "log", False, True, True, 0),
    (1, 300, 1, 1, 256, 40, BF16, "raw32", True, True, False, 4),
    (2, 192, 1, 3, 128, 16, BF16, "log", False, True, True, 0),
    (1, 150, 2, 2, 160, 48, F32, "raw", True, False, False, 0),
    (2, 129, 1, 1, 31, 129, BF16, "raw", True, True, True, 1),
    (1, 700, 1, 2, 128, 32, F32, "raw", True, True, False, 0),
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_delta(k):
    *shape, pad = CASES[k]
    x = case(Draw(500 + k), *shape)
    o, err, S, S_err = expected(x)
    dev = on_device(x, pad)
    got, end = ra.gated_delta(**dev)
    assert got.dtype == x["v"].dtype and end.dtype == F32
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")
    # Roundings are independent of each other: together they are off by the root of
    # their number, that of a sum over key_dim and of four over a chunk's steps, each
    # U at most (4: what earlier chunks left, which decays).
    for y, want in ((got, o), (end, S)):
        half = U if y.dtype == F32 else HALF_STEP[y.dtype]
        off = np.linalg.norm(y.cpu().double().numpy() - want)
        assert off <= (half + 4 * U * np.sqrt(shape[4] + 4 * 64)) * np.linalg.norm(want) + 1e-30
    lens = x["sequence_lens"]
    if lens is not None:
        for i, n in enumerate(lens.tolist()):
            assert not got[i, n:].contiguous().view(torch.int16 if got.dtype != F32 else torch.int32).any(), "not +0"
            if n == 0 and x["state"] is not None:
                assert torch.equal(end[i].cpu(), x["state"][i])
    # into a strided output, the state in place, the way without the compiled call: the same bits
    out = inside(torch.zeros_like(x["v"]), 5)
    hold = dev["state"].clone() if x["state"] is not None else torch.empty_like(end)
    more = dict(dev, state=hold) if x["state"] is not None else dev
    ra.gated_delta(**more, out=out, state_out=hold, stream=torch.cuda.current_stream())
    assert torch.equal(out, got) and torch.equal(hold, end)


def test_delta_in_parts_is_the_whole():
    x = case(Draw(7), 2, 230, 2, 4, 64, 48, F32, "log", False, True, False)
    o, err, S, S_err = expected(x)
    dev, outs, state = on_device(x), [], cuda(x["state"])
    for lo, hi in ((0, 1), (1, 3), (3, 70), (70, 70), (70, 199), (199, 230)):
        part = {n: dev[n][:, lo:hi] for n in ("q", "k", "v", "beta", "g")}
        y, state = ra.gated_delta(**part, state=state)
        outs.append(y)
    assert_close(torch.cat(outs, 1), o, 2 * err, "o")
    assert_close(state, S, 2 * S_err, "state")


@pytest.mark.parametrize("dtype,steps", [(F32, 1), (F32, 150), (BF16, 150), (F16, 5)])
def test_a_decay_to_nothing_forgets(dtype, steps):
    """-inf, and decays beyond float32: what came before leaves no trace."""
    r = Draw(11)
    x = case(r, 2, steps + 80, 1, 2, 64, 32, dtype, "log", True, True, False)
    at = steps - 1
    x["g"][0, at], x["g"][1, at] = -INF, -1e30
    x["g"][:, 3 + at] = -90.0
    o, err, S, S_err = expected(x)
    got, end = ra.gated_delta(**on_device(x))
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")
    fresh = {n: v[:, at:] if n in ("q", "k", "v", "beta", "g") else v for n, v in on_device(x).items()}
    fresh["g"] = fresh["g"].clone()
    fresh["state"] = None
    again, end2 = ra.gated_delta(**fresh)
    assert_close(again, got[:, at:].cpu().double().numpy(), err[:, at:] * 2, "o after")
    assert_close(end2, end.cpu().double().numpy(), S_err * 2, "state after")


def test_decays_above_nothing_count_as_none():
    x = case(Draw(12), 1, 90, 1, 1, 32, 32, F32, "log", True, True, False)
    x["g"].abs_()
    dev = on_device(x)
    a = ra.gated_delta(**dev)
    b = ra.gated_delta(**dict(dev, g=torch.zeros_like(dev["g"])))
    c = ra.gated_delta(**dict(dev, g=None))
    for p, q, s in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, s)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_keys(dtype):
    """The same key at every step, rates near 1: powers of the chunk's matrix
    exceed the inverse by many orders."""
    x = case(Draw(13), 1, 192, 1, 2, 64, 64, dtype, "log", False, False, False)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:] = 0.98 + 0.02 * x["beta"]
    x["g"][:] = x["g"] * 0.01
    o, err, S, S_err = expected(x)
    got, end = ra.gated_delta(**on_device(x))
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")


@pytest.mark.parametrize("steps", [1, 70])
def test_zero_keys_and_rates(steps):
    """No key, no rate: the state only decays; a query of zeros reads nothing."""
    x = case(Draw(14), 2, steps, 1, 1, 48, 20, BF16, "log", True, True, False)
    x["k"][0] = 0
    x["beta"][1] = 0
    x["q"][0] = 0
    o, err, S, S_err = expected(x)
    got, end = ra.gated_delta(**on_device(x))
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")
    assert not got[0].any()


@pytest.mark.parametrize("steps", [1, 100])
def test_what_is_not_finite_stays_in_its_row_and_column(steps):
    x = case(Draw(15), 3, steps, 2, 2, 64, 40, F32, "log", True, True, False)
    o, err, S, S_err = expected(x)
    at = steps // 2
    dev = on_device(x)
    dev["v"][1, at, 0, 7] = INF
    dev["k"][2, at, 0, 3] = NAN
    got, end = ra.gated_delta(**dev)
    assert_close(got[0], o[0], err[0], "row 0")
    assert_close(end[0], S[0], S_err[0], "row 0")
    # one value column of one head
    others = [c for c in range(40) if c != 7]
    assert_close(got[1][:, 0][:, others], o[1][:, 0][:, others], err[1][:, 0][:, others], "columns")
    assert_close(got[1][:, 1], o[1][:, 1], err[1][:, 1], "the other head")
    assert not torch.isfinite(got[1, at:, 0, 7]).any()
    # one head, whose chunk of 64 steps begins at 0: its later steps, not the other's
    assert got[2, at:, 0].isnan().all() and end[2, 0].isnan().all()
    assert_close(got[2][:, 1], o[2][:, 1], err[2][:, 1], "the other head")


def test_what_is_not_finite_leaves_earlier_chunks():
    x = case(Draw(22), 1, 200, 2, 2, 64, 40, BF16, "log", True, True, False)
    o, err, S, S_err = expected(x)
    dev = on_device(x)
    dev["q"][0, 130, 1, 5] = dev["k"][0, 140, 0, 3] = NAN
    got, end = ra.gated_delta(**dev)
    assert_close(got[:, :128], o[:, :128], err[:, :128], "o")
    assert got[0, 140:, 0].isnan().all() and got[0, 130, 1].isnan().all()
    # a query is read by its own step alone
    others = [t for t in range(200) if t != 130]
    assert_close(got[:, others][:, :, 1], o[:, others][:, :, 1], err[:, others][:, :, 1], "the other steps")
    assert_close(end[:, 1], S[:, 1], S_err[:, 1], "state")


def test_lengths_beyond_their_range_are_bounded():
    x = case(Draw(16), 3, 70, 1, 1, 32, 32, F32, "log", True, True, False)
    dev = on_device(x)
    lens = torch.tensor([-5, 99, 4], dtype=torch.int32).cuda()
    near = torch.tensor([0, 70, 4], dtype=torch.int32).cuda()
    for a, b in zip(ra.gated_delta(**dict(dev, sequence_lens=lens)),
                    ra.gated_delta(**dict(dev, sequence_lens=near))):
        assert torch.equal(a, b)


def test_nothing_to_do():
    x = case(Draw(17), 2, 5, 1, 2, 32, 16, BF16, "raw", True, True, False)
    dev = on_device(x)
    none = {n: dev[n][:, :0] for n in ("q", "k", "v", "beta", "g")}
    o, S = ra.gated_delta(**dict(dev, **none))
    assert o.shape == (2, 0, 2, 16) and torch.equal(S, dev["state"])
    o, S = ra.gated_delta(**dict(dev, **none, state=None))
    assert not S.any()
    none = {n: dev[n][:0] for n in ("q", "k", "v", "beta", "g", "state")}
    o, S = ra.gated_delta(**dict(dev, **none))
    assert o.shape == (0, 5, 2, 16) and S.shape == (0, 2, 32, 16)


@pytest.mark.parametrize("steps", [1, 130])
def test_captured_and_replayed(steps):
    x = case(Draw(18), 2, steps, 1, 2, 64, 64, BF16, "raw", True, True, True)
    dev = on_device(x)
    for n in ("q", "k", "v", "beta", "g"):
        dev[n] = torch.nan_to_num(dev[n])
    state = dev["state"].clone()
    want = []
    for _ in range(3):                  # the state moves on
        o, state = ra.gated_delta(**dict(dev, state=state))
        want.append((o, state))
    hold = dev["state"].clone()
    out = torch.empty_like(want[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.gated_delta(**dict(dev, state=hold), out=out, state_out=hold)
    hold.copy_(dev["state"])
    for o, s in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(hold, s)
        ra.gated_delta(**dev)           # eager work of the program's own between the replays
    # other lengths for the same graph
    hold.copy_(dev["state"])
    dev["sequence_lens"].copy_(torch.tensor([steps // 2, steps], dtype=torch.int32))
    o, s = ra.gated_delta(**dev)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(hold, s)


def test_on_another_stream_and_two_at_once():
    x = case(Draw(19), 2, 400, 2, 4, 128, 128, BF16, "raw", True, True, False)
    dev = on_device(x)
    want = ra.gated_delta(**dev)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [ra.gated_delta(**dev, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_rows_do_not_depend_on_each_other():
    x = case(Draw(20), 4, 150, 1, 2, 64, 64, BF16, "raw", True, True, True)
    dev = on_device(x)
    o, S = ra.gated_delta(**dev)
    for i in (0, 2):
        one = {n: v[i:i + 1] if n in ("q", "k", "v", "beta", "g", "state", "sequence_lens") else v
               for n, v in dev.items()}
        a, b = ra.gated_delta(**one)
        assert torch.equal(a[0], o[i]) and torch.equal(b[0], S[i])


def test_offsets_beyond_32_bits():
    """Steps 2^28 elements apart: offsets pass 2^32 bytes and 2^31 elements."""
    steps, stride = 20, 1 << 28
    x = case(Draw(21), 1, steps, 1, 1, 32, 32, BF16, "log", True, False, False)
    far_apart(x, steps, stride)


def far_apart(x, steps, stride):
    big = torch.empty(stride * (steps - 1) + 32 * 3, dtype=BF16, device="cuda")
    dev = on_device(x)
    for i, n in enumerate(("q", "k", "v")):
        view = big.as_strided((1, steps, 1, 32), (0, stride, 32, 1), 32 * i)
        view.copy_(dev[n])
        dev[n] = view
    got, end = ra.gated_delta(**dev)
    o, err, S, S_err = expected(x)
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")


@pytest.mark.parametrize("stride", [(1 << 24) - 65536 - 8, (1 << 24) - 65536])
def test_offsets_beyond_32_bits_in_chunks(stride):
    """The widest steps that chunks take (a chunk's rows within 2^31 bytes), and the first that they do not."""
    far_apart(case(Draw(22), 1, 300, 1, 1, 32, 32, BF16, "log", True, False, False), 300, stride)


def test_a_row_alone_is_as_in_a_batch():
    """Bit for bit, on either side of every rule on the number of heads."""
    for steps in (7, 12, 17, 40, 130):
        x = case(Draw(30 + steps), 24, steps, 2, 4, 64, 48, BF16, "raw", True, True, False)
        dev = on_device(x)
        o, S = ra.gated_delta(**dev)
        for i in (0, 23):
            one = {n: v[i:i + 1] if n in ("q", "k", "v", "beta", "g", "state") else v for n, v in dev.items()}
            a, b = ra.gated_delta(**one)
            assert torch.equal(a[0], o[i]) and torch.equal(b[0], S[i]), steps


WIDE = [  # more slices of 16 columns than compute units; batch, steps, key heads, heads, key dim, value dim, ...
    (6, 150, 4, 8, 128, 96, BF16, "raw", True, True, True, 0),
    (9, 70, 8, 8, 64, 72, F32, "log", False, True, True, 0),         # a last slice of 8
    (5, 129, 4, 8, 96, 100, F16, "raw", True, True, False, 8),       # of 4
    (17, 100, 4, 4, 40, 77, F32, "raw", True, False, True, 1),       # of 13
    (40, 65, 1, 2, 128, 49, BF16, "log", False, True, True, 1),
    (11, 90, 4, 8, 192, 56, BF16, "raw32", True, True, False, 0),
    (11, 66, 4, 8, 192, 47, F32, "log", True, True, True, 3),
    (11, 66, 8, 8, 256, 48, F16, "raw", True, True, True, 0),        # of keys too long for two slices
]


@pytest.mark.parametrize("k", range(len(WIDE)))
def test_many_heads(k):
    *shape, pad = WIDE[k]
    x = case(Draw(700 + k), *shape)
    o, err, S, S_err = expected(x)
    got, end = ra.gated_delta(**on_device(x, pad))
    assert_close(got, o, err, "o")
    assert_close(end, S, S_err, "state")


@pytest.mark.parametrize("dtype,ragged,b", [(BF16, False, 5), (F32, True, 2), (F16, False, 3)])
def test_more_chunks_than_are_prepared_at_once(dtype, ragged, b):
    """Parts of a sequence that each fit into the workspace are the sequence: every
    part goes on from the one before, also where a row has ended."""
    steps, h, d = 2300, 40, 128
    x = case(Draw(50), b, steps, h, h, d, d, dtype, "log", False, True, False)
    dev = on_device(x)
    if ragged:
        dev["sequence_lens"] = torch.tensor([900, steps], dtype=torch.int32, device="cuda")
    o, S = ra.gated_delta(**dev)
    # without a state at the end, which the parts between hand on all the same
    desc = _lib.rnn_delta_desc(batch=b, steps=steps, key_heads=h, heads=h, key_dim=d, value_dim=d,
                               dtype=(F32, BF16, F16).index(dtype), gate_dtype=(F32, BF16, F16).index(F32 if
                               dev["g"].dtype == F32 else dtype), scale=d ** -0.5)
    for n in "qkvo":
        setattr(desc, n + "_batch_stride", steps * h * d)
        setattr(desc, n + "_step_stride", h * d)
        setattr(desc, n + "_head_stride", d)
    for n in ("beta", "g"):
        setattr(desc, n + "_batch_stride", steps * h)
        setattr(desc, n + "_step_stride", h)
    size = ctypes.c_size_t()
    assert _lib.load().rnn_delta_workspace_size(ctypes.addressof(desc), ctypes.byref(size)) == 0
    assert size.value > 200 << 20
    space, other = torch.empty(size.value, dtype=torch.uint8, device="cuda"), torch.empty_like(o)
    at = {n: t.data_ptr() for n, t in dev.items() if isinstance(t, torch.Tensor)}
    assert _lib.load().rnn_delta_run(
        ctypes.addressof(desc), torch.cuda.current_stream().cuda_stream, space.data_ptr(), size.value, at["q"],
        at["k"], at["v"], at["beta"], at["g"], None, None, at["state"], at.get("sequence_lens"),
        other.data_ptr(), None) == 0
    assert torch.equal(other, o)
    parts, at, state = [], 0, dev["state"]
    while at < steps:
        n = min(512, steps - at)
        one = {k: v[:, at:at + n] if k in ("q", "k", "v", "beta", "g") else v for k, v in dev.items()}
        one["state"] = state
        if ragged:
            one["sequence_lens"] = (dev["sequence_lens"] - at).clamp(0, n).to(torch.int32)
        a, state = ra.gated_delta(**one)
        parts.append(a)
        at += n
    assert torch.equal(torch.cat(parts, 1), o) and torch.equal(state, S)
