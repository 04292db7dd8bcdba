"""The language-model operators on the GPU against their plain 64-bit
definitions (tests/lm_ref.py), within bounds that count the roundings of a
float32 evaluation; whole numbers exactly."""
import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from tests import lm_ref
from tests.lm_ref import U, assert_close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ra._lib.load()
    yield


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def normal(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.g) * (hi - lo) + lo

    def lens(self, batch, steps):
        n = torch.randint(0, steps + 1, (batch,), generator=self.g, dtype=torch.int32)
        n[0] = steps
        if batch > 1:
            n[-1] = 0
        return n


def cuda(t):
    return None if t is None else t.cuda()


def inside(t, pad, fill=NAN):
    """t as a view into a larger device tensor whose rest is `fill`."""
    big = torch.full((*t.shape[:-1], t.shape[-1] + 2 * pad), fill, dtype=t.dtype, device="cuda")
    view = big[..., pad:pad + t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# Convolution
# ---------------------------------------------------------------------------

CONV = [  # batch, steps, dim, taps, dtype, silu, bias, state, lens, pad
    (1, 1, 1, 1, F32, False, False, False, False, 0),
    (2, 1, 64, 4, BF16, True, True, True, False, 0),
    (3, 2, 64, 4, F16, True, True, True, True, 8),
    (1, 37, 24, 4, BF16, True, True, False, False, 0),
    (4, 37, 24, 4, BF16, True, False, True, True, 24),
    (5, 70, 17, 3, F32, False, True, True, True, 3),
    (2, 130, 40, 2, F16, True, True, True, True, 1),
    (3, 9, 33, 8, BF16, False, True, True, True, 0),
    (2, 65, 16, 5, F32, True, True, False, True, 4),
    (2, 20, 8, 6, F16, False, False, True, True, 0),
    (2, 20, 8, 7, F32, False, False, True, True, 0),
    (2, 257, 8, 1, BF16, True, True, False, True, 0),
    (1, 4100, 72, 4, BF16, True, True, True, False, 72),
]


@pytest.mark.parametrize("k", range(len(CONV)))
def test_conv(k):
    b, t, c, taps, dtype, silu, bias, state, lens, pad = CONV[k]
    r = Draw(100 + k)
    x, w = r.normal(b, t, c, dtype=dtype), r.normal(c, taps)
    bias = r.normal(c) if bias else None
    state = r.normal(b, taps - 1, c, dtype=dtype) if state else None
    lens = r.lens(b, t) if lens else None
    y, err, win = lm_ref.conv(x, w, bias, silu, state, lens)
    xd = inside(x, pad)
    if lens is not None:                # what a mask leaves out may hold anything
        for i, n in enumerate(lens.tolist()):
            xd[i, n:] = NAN
    got, gw = ra.causal_conv(xd, cuda(w), cuda(bias), silu=silu, state=cuda(state),
                             sequence_lens=cuda(lens))
    assert got.dtype == dtype and gw.dtype == dtype
    assert_close(got, y, err, "y")
    assert_close(gw, win, 0, "window")
    if lens is not None:
        for i, n in enumerate(lens.tolist()):
            assert not got[i, n:].view(torch.int16 if dtype != F32 else torch.int32).any(), "not +0"
    # into a strided output, and the window in place: the same bits
    out = inside(torch.zeros(b, t, c, dtype=dtype), 5)
    hold = cuda(state).clone() if state is not None else None
    ra.causal_conv(xd, cuda(w), cuda(bias), silu=silu, state=hold, sequence_lens=cuda(lens),
                   out=out, state_out=hold)
    assert torch.equal(out, got)
    if hold is not None:
        assert torch.equal(hold, gw)


def test_conv_in_parts_is_the_whole():
    r = Draw(7)
    x, w = r.normal(2, 50, 32, dtype=BF16).cuda(), r.normal(32, 4).cuda()
    whole, end = ra.causal_conv(x, w, silu=True)
    parts, win = [], None
    for lo, hi in ((0, 1), (1, 2), (2, 4), (4, 37), (37, 37), (37, 50)):
        y, win = ra.causal_conv(x[:, lo:hi], w, silu=True, state=win)
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(win, end)


def test_conv_lengths_beyond_their_range_are_bounded():
    r = Draw(8)
    x, w = r.normal(3, 10, 16).cuda(), r.normal(16, 3).cuda()
    lens = torch.tensor([-5, 99, 4], dtype=torch.int32).cuda()
    near = torch.tensor([0, 10, 4], dtype=torch.int32).cuda()
    for a, b in zip(ra.causal_conv(x, w, sequence_lens=lens),
                    ra.causal_conv(x, w, sequence_lens=near)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Scan
# ---------------------------------------------------------------------------

SCAN = [  # batch, steps, dim, states, groups, dtype, softplus, bias, skip, gate, state, lens, pad
    (1, 1, 1, 1, 1, F32, False, False, False, False, False, False, 0),
    (3, 1, 64, 16, 1, BF16, True, True, True, True, True, False, 0),
    (2, 1, 48, 16, 2, F32, True, True, True, True, True, False, 3),
    (2, 3, 40, 16, 1, F16, True, True, True, True, True, True, 8),
    (1, 16, 16, 16, 1, F32, True, True, True, False, True, False, 0),
    (2, 17, 32, 16, 1, F32, True, True, True, True, False, False, 0),
    (3, 100, 32, 16, 2, F32, True, True, True, True, True, True, 16),
    (2, 129, 20, 13, 1, F32, False, True, False, True, True, True, 1),
    (2, 70, 12, 64, 3, F32, True, False, True, True, True, True, 0),
    (2, 70, 12, 33, 1, F32, True, True, True, False, True, True, 5),
    (2, 90, 24, 8, 2, BF16, True, True, True, True, True, True, 8),
    (2, 90, 24, 4, 1, F32, True, True, True, True, True, True, 0),
    (1, 65, 17, 3, 1, F16, True, True, False, False, True, False, 2),
    (1, 1500, 16, 16, 1, F32, True, True, True, True, True, False, 0),
    (1, 1501, 33, 5, 1, F32, True, True, True, True, False, False, 0),
    (2, 2048, 8, 16, 1, BF16, True, True, True, True, True, True, 0),
    (9, 40, 400, 16, 1, BF16, True, True, True, True, True, True, 0),
]


def scan_inputs(r, b, t, c, n, g, dtype, softplus, bias, skip, gate, state, lens):
    step = r.uniform(b, t, c, lo=0.001, hi=0.3)
    v = {"x": r.normal(b, t, c, dtype=dtype),
         "dt": (torch.log(torch.expm1(step)) if softplus else step).to(dtype),
         "A": -r.uniform(c, n, lo=0.2, hi=1.0) * torch.arange(1, n + 1),
         "B": r.normal(b, t, g, n, dtype=dtype), "C": r.normal(b, t, g, n, dtype=dtype),
         "D": r.normal(c) if skip else None, "z": r.normal(b, t, c, dtype=dtype) if gate else None,
         "dt_bias": r.normal(c, scale=0.3) if bias and softplus else
         r.uniform(c, hi=0.1) if bias else None,
         "state": r.normal(b, c, n) if state else None, "lens": r.lens(b, t) if lens else None}
    if g == 1:
        v["B"], v["C"] = v["B"][:, :, 0], v["C"][:, :, 0]
    return v


def scan_call(v, softplus, pad=0, **more):
    p = {k: inside(v[k], pad) if v[k] is not None else None for k in ("x", "dt", "B", "C", "z")}
    if v["lens"] is not None:           # what a mask leaves out may hold anything
        for i, n in enumerate(v["lens"].tolist()):
            for k, bad in zip(p, (NAN, INF, -INF, NAN, INF)):
                if p[k] is not None:
                    p[k][i, n:] = bad
    kw = dict(D=cuda(v["D"]), z=p["z"], dt_bias=cuda(v["dt_bias"]), dt_softplus=softplus,
              state=cuda(v["state"]), sequence_lens=cuda(v["lens"]))
    kw.update(more)
    return ra.selective_scan(p["x"], p["dt"], cuda(v["A"]), p["B"], p["C"], **kw)


@pytest.mark.parametrize("k", range(len(SCAN)))
def test_scan(k):
    *spec, pad = SCAN[k]
    b, t, c, n, g, dtype, softplus = spec[:7]
    v = scan_inputs(Draw(200 + k), *spec)
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], softplus, v["state"], v["lens"])
    got, gh = scan_call(v, softplus, pad)
    assert got.dtype == dtype and gh.dtype == F32
    assert_close(got, y, err, "y")
    assert_close(gh, h, herr, "state")
    if v["lens"] is not None:
        for i, m in enumerate(v["lens"].tolist()):
            assert not got[i, m:].view(torch.int16 if dtype != F32 else torch.int32).any(), "not +0"
            if m == 0 and v["state"] is not None:
                assert torch.equal(gh[i].cpu(), v["state"][i])
    # into a strided output, the state in place: the same bits
    out = inside(torch.zeros(b, t, c, dtype=dtype), 5)
    hold = cuda(v["state"]).clone() if v["state"] is not None else None
    scan_call(v, softplus, pad, state=hold, out=out, state_out=hold)
    assert torch.equal(out, got)
    if hold is not None:
        assert torch.equal(hold, gh)


def test_scan_single_tokens_follow_the_prompt():
    spec = (2, 70, 32, 16, 1, F32, True, True, True, True, True, False)
    v = scan_inputs(Draw(301), *spec)
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], True, v["state"], None)
    part = lambda lo, hi: {k: (w[:, lo:hi] if k in ("x", "dt", "B", "C", "z") else w)  # noqa: E731
                           for k, w in v.items()}
    got, state = scan_call(part(0, 60), True)
    parts = [got]
    for i in range(60, 70):
        got, state = scan_call(part(i, i + 1), True, state=state)
        parts.append(got)
    assert_close(torch.cat(parts, 1), y, err, "y")
    assert_close(state, h, herr, "state")


def test_scan_infinite_and_nan_inputs_stay_in_their_rows():
    spec = (3, 40, 16, 13, 1, F32, True, True, True, False, True, False)
    v = scan_inputs(Draw(302), *spec)
    clean, _ = scan_call(v, True)
    v["x"][1, 7, 3] = NAN
    v["x"][2, 9, 5] = INF
    got, _ = scan_call(v, True)
    same = torch.ones(3, 40, 16, dtype=torch.bool)
    same[1, 7:, 3] = False
    same[2, 9:, 5] = False
    assert torch.equal(got.cpu()[same], clean.cpu()[same])
    assert torch.isnan(got[1, 7:, 3]).all() and not torch.isfinite(got[2, 9, 5])


def test_scan_softplus_over_its_range():
    # y = step size itself: x = B = C = 1, A = 0, one step
    raw = torch.cat([torch.linspace(-90, 90, 4001), torch.tensor([-INF, INF, NAN, 0.0, -0.0])])
    n = raw.numel()
    one = torch.ones(1, 1, n)
    got, _ = ra.selective_scan(one.cuda(), raw.view(1, 1, n).cuda(), torch.zeros(n, 1).cuda(),
                               torch.ones(1, 1, 1).cuda(), torch.ones(1, 1, 1).cuda(),
                               dt_softplus=True)
    with np.errstate(all="ignore"):
        want = np.logaddexp(0, raw.double().numpy())
        want = np.exp(want * 0) * 0 + want      # the step's decay of the zero state: NaN where it is
        err = want * (2 * np.abs(raw.double().numpy()) + 24) * U + 2.0 ** -126
    assert_close(got[0, 0], want, np.where(np.isfinite(err), err, 0), "softplus")


def test_scan_zero_steps_hand_the_state_on():
    h = torch.randn(2, 8, 16).cuda()
    e = torch.empty(2, 0, 8).cuda()
    s = torch.empty(2, 0, 16).cuda()
    y, got = ra.selective_scan(e, e, torch.zeros(8, 16).cuda(), s, s, state=h)
    assert y.shape == (2, 0, 8) and torch.equal(got, h)
    _, got = ra.selective_scan(e, e, torch.zeros(8, 16).cuda(), s, s)
    assert not got.any()


# ---------------------------------------------------------------------------
# 8-bit rows and their product
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (1, 1, F32, 0), (3, 16, BF16, 0), (5, 100, F16, 3), (7, 128, F32, 4), (2, 1000, BF16, 8),
    (33, 2501, F32, 0), (4, 4096, BF16, 0), (2, 8200, F16, 8), (3, 20000, BF16, 0),
    (2, 40000, F32, 1)])
def test_quantize_rows(rows, cols, dtype, pad):
    r = Draw(rows * 7919 + cols)
    x = r.normal(rows, cols, dtype=dtype)
    if rows > 2:
        x[1] = 0
    if rows > 4:
        x[2, cols // 2] = INF
        x[3, cols - 1] = NAN
        x[4] = x[4].float() * (2.0 ** -20 if dtype == F16 else 2.0 ** -110)
    q, scale = lm_ref.quantize(x)
    got = ra.quantize_rows(inside(x, pad))
    assert np.array_equal(got.q.cpu().numpy(), q)
    assert np.array_equal(got.scale.cpu().numpy(), scale, equal_nan=True)
    assert got.q.stride(0) % 128 == 0
    full = got.q.as_strided((rows, got.q.stride(0)), (got.q.stride(0), 1))
    assert not full[:, cols:].any()


PROJECT = [  # rows, cols, outs, dtype, bias, pad
    (1, 1, 1, F32, False, 0), (1, 64, 32, BF16, False, 0), (1, 2048, 1000, BF16, True, 0),
    (4, 500, 333, F16, True, 4), (16, 256, 100, F32, False, 0), (17, 256, 130, F32, True, 0),
    (33, 130, 65, BF16, True, 3), (64, 1024, 512, BF16, False, 8), (100, 77, 300, F16, False, 0),
    (255, 1500, 257, F32, True, 0), (300, 640, 777, BF16, True, 0), (513, 384, 1024, F16, True, 0),
    (2, 20000, 48, F32, True, 0), (130, 9000, 40, F32, True, 0), (8, 4096, 4096, BF16, True, 0),
    (1025, 192, 520, BF16, False, 0),
]


def weights(r, outs, cols, pitch=None):
    w = torch.randint(-127, 128, (outs, cols), generator=r.g, dtype=torch.int8)
    pitch = pitch or (cols + 15) // 16 * 16
    # what lies past the columns may hold anything
    full = torch.randint(-127, 128, (outs, pitch), generator=r.g, dtype=torch.int8)
    full[:, :cols] = w
    return w, full.cuda()[:, :cols], r.uniform(outs, lo=0.5, hi=1.5) / (73 * cols ** 0.5)


@pytest.mark.parametrize("k", range(len(PROJECT)))
def test_project(k):
    rows, cols, outs, dtype, bias, pad = PROJECT[k]
    r = Draw(400 + k)
    x = r.normal(rows, cols, dtype=dtype)
    if rows > 3:
        x[2] = 0
    w, wd, ws = weights(r, outs, cols)
    bias = r.normal(outs) if bias else None
    q, scale = lm_ref.quantize(x)
    y, err = lm_ref.project(q, scale, w, ws, bias, dtype)
    xd = inside(x, pad)
    got = ra.quant_project(xd, wd, ws.cuda(), bias=cuda(bias))
    assert got.dtype == dtype
    assert_close(got, y, err, "y")
    # rows that are 8-bit already, a strided output, another type
    rowsq = ra.quantize_rows(xd)
    again = ra.quant_project(rowsq.q, wd, ws.cuda(), bias=cuda(bias), x_scale=rowsq.scale,
                             out=inside(torch.zeros(rows, outs, dtype=dtype), 3))
    assert torch.equal(again, got)
    wide = ra.quant_project(xd, wd, ws.cuda(), bias=cuda(bias), out_dtype=F32)
    y, err = lm_ref.project(q, scale, w, ws, bias, F32)
    assert_close(wide, y, err, "y in float32")


def test_project_sums_are_exact_at_the_largest_size():
    cols = ra._lib.RNN_QUANT_MAX_COLS
    for rows in (1, 40):
        q = torch.full((rows, 131072), -128, dtype=torch.int8).cuda()
        q[:, cols:] = 0
        w = torch.full((3, 131072), -128, dtype=torch.int8).cuda()
        w[1] = 127
        w[2] = 1
        one = torch.ones(3).cuda()
        y = ra.quant_project(q[:, :cols], w[:, :cols], one, x_scale=torch.ones(rows).cuda())
        for o, v in enumerate((128, -127, -1)):
            assert (y[:, o] == float(np.float32(128 * v * cols))).all()


def test_project_rows_that_are_not_finite_give_nan_alone():
    r = Draw(11)
    for rows in (3, 70):
        x = r.normal(rows, 200)
        _, wd, ws = weights(r, 64, 200)
        clean = ra.quant_project(x.cuda(), wd, ws.cuda())
        x[1, 5] = INF
        x[rows - 1, 199] = NAN
        got = ra.quant_project(x.cuda(), wd, ws.cuda())
        bad = torch.zeros(rows, dtype=torch.bool)
        bad[1] = bad[rows - 1] = True
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


def test_project_no_columns_is_the_bias():
    x = torch.empty(3, 0).cuda()
    w = torch.empty(5, 16, dtype=torch.int8).cuda()[:, :0]
    b = torch.arange(5.0).cuda()
    assert torch.equal(ra.quant_project(x, w, torch.ones(5).cuda(), bias=b), b.expand(3, 5))
    assert ra.quant_project(x[:0], w, torch.ones(5).cuda()).shape == (0, 5)


# ---------------------------------------------------------------------------
# Token scores
# ---------------------------------------------------------------------------

def check_scores(logits, tokens, top, pad=0):
    want = lm_ref.scores(logits, tokens, top)
    got = ra.token_scores(inside(logits, pad), cuda(tokens), top=top)
    err = want["err"]
    assert np.array_equal(got.top_ids.cpu().numpy(), want["top_ids"])
    with np.errstate(invalid="ignore"):
        assert_close(got.top_logprobs, want["top_logprobs"],
                     err[:, None] + 4 * U * np.abs(want["top_logprobs"]), "top_logprobs")
        assert_close(got.entropy, want["entropy"], want["err_entropy"], "entropy")
        if tokens is None:
            assert got.logprob is None and got.rank is None
            return got
        assert np.array_equal(got.rank.cpu().numpy(), want["rank"])
        assert_close(got.logprob, want["logprob"], err + 4 * U * np.abs(want["logprob"]), "logprob")
    return got


SCORES = [  # rows, vocab, top, dtype, token type, pad, kind
    (1, 1, 1, F32, torch.int64, 0, "normal"), (2, 3, 5, BF16, torch.int32, 0, "normal"),
    (3, 100, 0, F32, torch.int32, 1, "normal"), (5, 1000, 64, F16, torch.int64, 3, "normal"),
    (4, 5000, 20, BF16, torch.int64, 8, "normal"), (2, 70001, 8, F32, torch.int64, 0, "masked"),
    (1, 131072, 32, BF16, torch.int64, 0, "normal"), (40, 4097, 33, F16, torch.int32, 0, "masked"),
    (300, 2000, 5, BF16, torch.int64, 0, "normal"), (2, 200000, 20, BF16, torch.int64, 0, "masked"),
    (3, 30000, 20, F32, torch.int64, 0, "rising"), (3, 30000, 64, BF16, torch.int64, 0, "rising"),
    (3, 30000, 20, F32, torch.int64, 0, "falling"), (4, 9000, 64, F32, torch.int64, 0, "equal"),
    (4, 9000, 64, BF16, torch.int64, 0, "few"), (2, 100000, 64, F32, torch.int64, 0, "late"),
]


@pytest.mark.parametrize("k", range(len(SCORES)))
def test_scores(k):
    rows, vocab, top, dtype, ints, pad, kind = SCORES[k]
    r = Draw(500 + k)
    x = r.normal(rows, vocab, scale=3.0)
    if kind == "masked":
        x[r.uniform(rows, vocab) < 0.7] = -INF
        x[0, :vocab // 2] = -INF
    elif kind == "rising":
        x = torch.linspace(-20, 20, vocab).repeat(rows, 1)
    elif kind == "falling":
        x = torch.linspace(20, -20, vocab).repeat(rows, 1)
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "few":                 # fewer entries left than alternatives
        keep = torch.zeros(vocab, dtype=torch.bool)
        keep[[3, 77, 4000, vocab - 1]] = True
        x[:, ~keep] = -INF
    elif kind == "late":                # everything that counts at the end
        x[:, :vocab - 100] -= 50
    x = x.to(dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=r.g).to(ints)
    tokens[0] = vocab - 1
    if rows > 1:
        tokens[1] = int(x[1].float().argmax())
    check_scores(x, tokens, top, pad)


def test_scores_edges():
    x = torch.randn(9, 300, generator=torch.Generator().manual_seed(2))
    x[0] = -INF                      # a mask that leaves nothing
    x[1, 7] = INF
    x[2, 9] = NAN
    x[3] = 0.0
    x[3, ::2] = -0.0                 # equal zeros of both signs
    x[4, 5], x[4, 200] = NAN, -NAN
    x[5] = torch.finfo(F32).min      # a mask of the lowest value
    x[6, 1:] = torch.finfo(F32).min
    x[7] *= 1e30
    tokens = torch.tensor([3, 7, 10, 5, 200, 100, 0, 8, 12])
    check_scores(x, tokens, 10)
    check_scores(x, None, 3)
    check_scores(x, torch.tensor([-1, 300, 1 << 40, 0, 1, 2, 3, 4, 5]), 2)
    check_scores(x, torch.tensor([9, 9, 9, 9, 9, 9, 9, 9, 9], dtype=torch.int32), 0)


def test_scores_rows_apart_in_memory():
    # offsets past 32 bits: rows 3 GiB apart
    stride = 3 * (1 << 30) // 2
    big = torch.empty(stride + 5000, dtype=BF16, device="cuda")
    x = big.as_strided((2, 5000), (stride, 1))
    v = torch.randn(2, 5000, generator=torch.Generator().manual_seed(4)).to(BF16)
    x.copy_(v)
    want = ra.token_scores(v.cuda(), torch.tensor([4, 9]).cuda(), top=7)
    got = ra.token_scores(x, torch.tensor([4, 9]).cuda(), top=7)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Streams, graphs, refusals
# ---------------------------------------------------------------------------

def all_calls(r, b=3, t=40, c=64, n=16):
    """One call of each operator on inputs of its own, as a function of a
    stream; and the inputs."""
    v = scan_inputs(r, b, t, c, n, 1, BF16, True, True, True, True, True, True)
    v = {k: cuda(w) for k, w in v.items()}
    w4, x2 = r.normal(c, 4).cuda(), r.normal(50, 200, dtype=BF16).cuda()
    _, wd, ws = weights(r, 96, 200)
    ws = ws.cuda()
    lg, tk = r.normal(5, 60000).cuda(), torch.arange(5).cuda()

    def go(stream=None):
        y, win = ra.causal_conv(v["x"], w4, silu=True, sequence_lens=v["lens"], stream=stream)
        s, h = ra.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                                 dt_bias=v["dt_bias"], dt_softplus=True, state=v["state"],
                                 sequence_lens=v["lens"], stream=stream)
        q = ra.quantize_rows(x2, stream=stream)
        p = ra.quant_project(x2, wd, ws, stream=stream)
        p1 = ra.quant_project(x2[:2], wd, ws, stream=stream)
        return (y, win, s, h, *q, p, p1, *ra.token_scores(lg, tk, top=5, stream=stream))

    return go, (v, x2, lg)


def test_another_stream_gives_the_same():
    go, _ = all_calls(Draw(600))
    want = go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = go(side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_a_captured_graph_replays_with_new_inputs():
    go, (v, x2, lg) = all_calls(Draw(601))
    go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = go()
    for k in range(4):
        r = Draw(610 + k)
        v["x"].copy_(r.normal(*v["x"].shape, dtype=BF16))
        v["lens"].copy_(r.lens(3, 40))
        x2.copy_(r.normal(*x2.shape, dtype=BF16))
        lg.copy_(r.normal(*lg.shape))
        want = [o.clone() for o in go()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_twice_the_same_bits():
    go, _ = all_calls(Draw(602), t=700)
    for a, b in zip(go(), go()):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    x, w = torch.zeros(2, 5, 8).cuda(), torch.zeros(8, 4).cuda()
    h = torch.zeros(2, 8, 4).cuda()
    A, B = torch.zeros(8, 4).cuda(), torch.zeros(2, 5, 4).cuda()
    lens = torch.tensor([5, 5], dtype=torch.int32).cuda()
    bad = [
        lambda: ra.causal_conv(x, w.double()), lambda: ra.causal_conv(x, w[:4]),
        lambda: ra.causal_conv(x, w.cpu()), lambda: ra.causal_conv(x, w, torch.zeros(7).cuda()),
        lambda: ra.causal_conv(x, w, state=torch.zeros(2, 4, 8).cuda()),
        lambda: ra.causal_conv(x, w, state=torch.zeros(2, 3, 8).cuda().bfloat16()),
        lambda: ra.causal_conv(x, w, sequence_lens=lens.long()),
        lambda: ra.causal_conv(x, w, sequence_lens=[6, 1]),
        lambda: ra.causal_conv(x.transpose(1, 2), w), lambda: ra.causal_conv(x[0], w),
        lambda: ra.causal_conv(x.double(), w), lambda: ra.causal_conv(x, w, out=x[:, :4]),
        lambda: ra.selective_scan(x, x.bfloat16(), A, B, B),
        lambda: ra.selective_scan(x, x, A, B, B[:, :, :3]),
        lambda: ra.selective_scan(x, x, A[:, :3], B, B),
        lambda: ra.selective_scan(x, x, A.t().contiguous().t(), B, B),
        lambda: ra.selective_scan(x, x, A, B, B, state=h.bfloat16()),
        lambda: ra.selective_scan(x, x, A, B, B, z=x[:, :4]),
        lambda: ra.quantize_rows(x), lambda: ra.quantize_rows(x[0].t()),
        lambda: ra.quant_project(x[0], torch.zeros(6, 7, dtype=torch.int8).cuda(), w[:6, 0]),
        lambda: ra.quant_project(x[0], torch.zeros(6, 8).cuda(), torch.zeros(6).cuda()),
        lambda: ra.quant_project(x[0], torch.zeros(6, 8, dtype=torch.int8).cuda(),
                                 torch.zeros(6).cuda(), x_scale=torch.zeros(5).cuda()),
        lambda: ra.quant_project(x[0].char(), torch.zeros(6, 8, dtype=torch.int8).cuda(),
                                 torch.zeros(6).cuda()),
        lambda: ra.token_scores(x[0], lens), lambda: ra.token_scores(x[0], torch.zeros(5).cuda()),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"accepted: {k}")
    refused = [
        lambda: ra.causal_conv(x, torch.zeros(8, 9).cuda()),
        lambda: ra.causal_conv(x, w, out=x),
        lambda: ra.selective_scan(x, x, torch.zeros(8, 65).cuda(), *[torch.zeros(2, 5, 65).cuda()] * 2),
        lambda: ra.selective_scan(x, x, A, *[torch.zeros(2, 5, 3, 4).cuda()] * 2),
        lambda: ra.quant_project(x[0], torch.zeros(6, 8, dtype=torch.int8).cuda(),
                                 torch.zeros(6).cuda()),
        lambda: ra.token_scores(x[0], top=65), lambda: ra.token_scores(x[0], top=-1),
        lambda: ra.token_scores(x[0][:, :0]),
    ]
    for call in refused:
        with pytest.raises(ra.RNNError) as e:
            call()
        assert e.value.status == ra.RNN_ERR_INVALID_INPUT
