"""The language-model operators where their kernels change form: every tile of
the projection with columns and rows that end inside it, few rows beside many
weights, spans of the scan, channel groups that fill no workgroup, states in
place; against the plain 64-bit definitions (tests/lm_ref.py), or, where those
would take long, against exact integer arithmetic."""
import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from tests import lm_ref
from tests.lm_ref import assert_close
from tests.test_gpu_lm import (BF16, F16, F32, INF, NAN, Draw, _gpu, check_scores, cuda,  # noqa: F401
                               inside, scan_call, scan_inputs, weights)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,outs,dtype", [
    (2048, 96, 6144 + 7, F32),         # 256 x 256 tiles, a step and a half of columns
    (3500, 335, 3600, BF16),
    (4096, 64, 4096, F16), (1700, 272, 1500, F32),      # 128 x 128
    (900, 500, 1500, BF16),            # 64 x 64, more than 256
    (70, 255, 70, F32), (70, 256, 70, F16), (70, 257, 70, BF16), (90, 1040, 33, F32),
    (17, 3000, 129, F32), (500, 16, 200, BF16)])         # columns among the waves
def test_projection_tiles(rows, cols, outs, dtype):
    r = Draw(rows + 3 * cols + 7 * outs)
    q = torch.randint(-127, 128, (rows, cols), generator=r.g, dtype=torch.int8)
    x = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8)
    x[:, :cols] = q
    w, wd, ws = weights(r, outs, cols)
    xs, bias = r.uniform(rows, lo=0.5, hi=1.5), r.normal(outs)
    got = ra.quant_project(x.cuda()[:, :cols], wd, ws.cuda(), bias=bias.cuda(), x_scale=xs.cuda(),
                           out_dtype=dtype)
    # in 64 bits: the sums pass 2^24
    total = (q.cuda().double() @ w.cuda().double().t()).cpu().numpy()
    y = total * xs.double().numpy()[:, None] * ws.double().numpy()
    err = 4 * lm_ref.U * np.abs(y)
    y = y + bias.double().numpy()
    assert_close(got, y, lm_ref.stored(y, 2 * (err + 2 * lm_ref.U * np.abs(y)), dtype), "y")


@pytest.mark.parametrize("rows,cols,outs,dtype", [
    (1700, 176, 3900, F32), (2040, 64, 4095, BF16), (1930, 1000, 3973, F16),    # 256 x 128
    (500, 96, 3970, BF16), (385, 63, 4090, F32), (512, 1234, 3333, F16)])       # 128 x 64
def test_projection_oblong_tiles(rows, cols, outs, dtype):
    test_projection_tiles(rows, cols, outs, dtype)


@pytest.mark.parametrize("rows", [1, 3, 16])
def test_projection_of_few_rows_and_many_weights(rows):
    r = Draw(rows)
    cols, outs = 4100, 16400                   # more than 64 MiB of them
    q = torch.randint(-127, 128, (rows, cols), generator=r.g, dtype=torch.int8)
    x = torch.zeros(rows, 4112, dtype=torch.int8)
    x[:, :cols] = q
    w, wd, ws = weights(r, outs, cols)
    got = ra.quant_project(x.cuda()[:, :cols], wd, ws.cuda(), x_scale=torch.ones(rows).cuda())
    total = (q.double() @ w.double().t()).numpy()
    y = total * ws.double().numpy()
    assert_close(got, y, lm_ref.stored(y, 8 * lm_ref.U * np.abs(y), F32), "y")


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 16384), (2, 8192), (16, 1024), (16, 1000), (5, 3),
                                       (16, 1025), (3, 5462)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_rounded_inside_are_the_rounded_rows(rows, cols, dtype):
    r = Draw(rows * cols)
    x = r.normal(rows, cols, dtype=dtype)
    if rows > 2:
        x[1] = 0
        x[2, cols - 1] = INF
    _, wd, ws = weights(r, 40, cols)
    q = ra.quantize_rows(x.cuda())
    want = ra.quant_project(q.q, wd, ws.cuda(), x_scale=q.scale, out_dtype=dtype)
    got = ra.quant_project(inside(x, 3), wd, ws.cuda())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
    assert rows <= 2 or torch.isnan(got[2]).all()


@pytest.mark.parametrize("cols", [1, 7, 16, 31, 127, 128, 129, 500, 512, 513, 2047, 2048, 2049, 8193,
                                  32768, 32769, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rounding_of_rows_of_every_length(cols, dtype):
    r = Draw(cols)
    x = r.normal(67, cols, dtype=dtype)
    x[3] = 0
    x[5, cols - 1], x[6, cols // 2] = NAN, -INF
    x[7, cols - 1] = 100.0                  # the largest is the last one
    want_q, want_scale = lm_ref.quantize(x)
    got = ra.quantize_rows(inside(x, 1))
    assert np.array_equal(got.q.cpu().numpy(), want_q)
    assert np.array_equal(got.scale.cpu().numpy(), want_scale, equal_nan=True)


SPANS = [  # batch, steps, dim, states, groups, dtype, softplus, bias, skip, gate, state, lens
    (1, 900, 16, 16, 1, F32, True, True, True, True, True, False),
    (3, 700, 20, 16, 1, F32, True, True, True, True, True, True),
    (2, 1000, 30, 7, 2, F32, True, True, False, False, True, True),
    (1, 1200, 24, 40, 3, F32, True, True, True, True, False, False),
    (2, 800, 16, 64, 1, BF16, True, True, True, True, True, True),
    (2, 640, 33, 48, 11, F32, False, False, True, False, True, True),
]


@pytest.mark.parametrize("k", range(len(SPANS)))
def test_scan_in_spans(k):
    spec = SPANS[k]
    v = scan_inputs(Draw(900 + k), *spec)
    if v["lens"] is not None:              # one that ends at a span's border, one within the first
        v["lens"][1:] = torch.tensor([128, 5][:len(v["lens"]) - 1])
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], spec[6], v["state"], v["lens"])
    got, gh = scan_call(v, spec[6])
    assert_close(got, y, err, "y")
    assert_close(gh, h, herr, "state")
    if v["state"] is not None:             # the state in place, while spans read it
        hold = cuda(v["state"]).clone()
        again, _ = scan_call(v, spec[6], state=hold, state_out=hold)
        assert torch.equal(again, got) and torch.equal(hold, gh)


@pytest.mark.parametrize("steps", [1, 8, 9, 15, 16, 63, 64, 65, 127])
@pytest.mark.parametrize("states", [16, 5])
def test_scan_lengths_around_its_tiles(steps, states):
    spec = (2, steps, 19, states, 1, F32, True, True, True, True, True, True)
    v = scan_inputs(Draw(steps), *spec)
    v["lens"][1] = steps // 2
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], True, v["state"], v["lens"])
    got, gh = scan_call(v, True)
    assert_close(got, y, err, "y")
    assert_close(gh, h, herr, "state")


# Channels of a group and states of which four adjacent ones are loaded at once,
# where the last workgroup's and the last four are moved.
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("per,states", [(16, 4), (17, 5), (31, 6), (19, 7), (18, 18), (33, 35),
                                        (47, 49), (20, 62), (15, 6), (17, 3)])
def test_scan_of_odd_channels_and_states(per, states, dtype):
    spec = (2, 150, 2 * per, states, 2, dtype, True, True, True, True, True, True)
    v = scan_inputs(Draw(per + states), *spec)
    v["lens"][0] = 150
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], True, v["state"], v["lens"])
    got, gh = scan_call(v, True, pad=1)
    assert_close(got, y, err, "y")
    assert_close(gh, h, herr, "state")
    hold = cuda(v["state"]).clone()
    again, _ = scan_call(v, True, pad=1, state=hold, state_out=hold)
    assert torch.equal(again, got) and torch.equal(hold, gh)


# Many rows, short prompts: as the workgroups fill the chip, the states stay in
# registers for more steps.  (A group of one channel each is a workgroup.)
@pytest.mark.parametrize("batch,steps,states", [
    (4, 16, 16), (4, 17, 13), (8, 32, 6), (8, 33, 6), (16, 64, 8), (16, 65, 8), (16, 40, 9)])
def test_scan_of_many_short_rows(batch, steps, states):
    spec = (batch, steps, 256, states, 256, F32, True, True, True, True, True, True)
    v = scan_inputs(Draw(batch + steps), *spec)
    y, err, h, herr = lm_ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"],
                                  v["dt_bias"], True, v["state"], v["lens"])
    got, gh = scan_call(v, True)
    assert_close(got, y, err, "y")
    assert_close(gh, h, herr, "state")


@pytest.mark.parametrize("states", [16, 13, 40])
def test_scan_infinities_keep_to_their_channel_and_time(states):
    spec = (1, 200, 48, states, 1, F32, True, True, True, True, True, False)
    v = scan_inputs(Draw(77), *spec)
    clean, _ = scan_call(v, True)
    v["x"][0, 70, 20] = -INF
    got, state = scan_call(v, True)
    bad = torch.zeros(1, 200, 48, dtype=torch.bool)
    bad[0, 70:, 20] = True
    assert torch.equal(got.cpu()[~bad], clean.cpu()[~bad])
    assert not torch.isfinite(got[0, 70, 20]) and torch.isfinite(state[0, :20]).all()


def test_convolution_of_odd_channels_with_its_window_in_place():
    r = Draw(5)
    for dim in (1, 2, 3, 5, 7, 33):
        for dtype in (F32, BF16):
            x, w = r.normal(3, 40, dim, dtype=dtype), r.normal(dim, 4)
            state = r.normal(3, 3, dim, dtype=dtype)
            y, err, win = lm_ref.conv(x, w, None, True, state, None)
            hold = state.cuda()
            got, _ = ra.causal_conv(inside(x, 1), w.cuda(), silu=True, state=hold, state_out=hold)
            assert_close(got, y, err, "y")
            assert_close(hold, win, 0, "window")


@pytest.mark.parametrize("steps", [5, 8, 9, 16, 40])
def test_convolution_with_its_window_in_place_and_many_runs(steps):
    r = Draw(steps)
    x, w = r.normal(70, steps, 260).cuda(), r.normal(260, 8).cuda()
    state = r.normal(70, 7, 260).cuda()
    want, window = ra.causal_conv(x, w, state=state)
    hold = state.clone()
    got, _ = ra.causal_conv(x, w, state=hold, state_out=hold)
    assert torch.equal(got, want) and torch.equal(hold, window)


@pytest.mark.parametrize("rows,vocab,top,dtype", [
    (1, 262144, 64, F32), (1, 8193, 3, BF16), (2, 16391, 64, F16), (7, 65539, 1, BF16),
    (520, 9001, 20, F32), (3, 8, 8, F32), (3, 7, 2, BF16), (2, 2049, 64, F32)])
def test_scores_in_segments_and_odd_ends(rows, vocab, top, dtype):
    r = Draw(vocab + top)
    x = r.normal(rows, vocab, scale=3.0, dtype=dtype)
    x[0, -1] = 20.0                         # the best entry is the last one
    tokens = torch.randint(0, vocab, (rows,), generator=r.g)
    tokens[0] = vocab - 1
    check_scores(x, tokens, top, pad=1)


def test_scores_of_equal_entries_over_segments():
    x = torch.zeros(2, 70001)
    x[1, 40000:] = 1.0
    x[1, 69990] = NAN
    check_scores(x, torch.tensor([70000, 69990]), 64)
    y = torch.full((3, 70001), -INF)        # a mask that leaves one, two, no entries
    y[0, 69999] = -3.0
    y[1, 5] = y[1, 60000] = 2.0
    check_scores(y, torch.tensor([69999, 60000, 4]), 20)
    check_scores(y.to(BF16), torch.tensor([5, 5, 70000]), 5)


@pytest.mark.parametrize("vocab", [1, 7, 8, 9, 65, 129, 500, 511, 512, 513, 1000, 1024, 1025, 2041,
                                   2047, 2048, 2049])
@pytest.mark.parametrize("top,dtype", [(0, F16), (1, F32), (20, BF16), (64, F16), (64, F32)])
def test_scores_of_short_rows(vocab, top, dtype):
    r = Draw(vocab + top)
    x = r.normal(14, vocab, scale=3.0)
    x[1] = 0.5                              # equal entries
    x[2, vocab // 2:] = 7.0                 # the best ones equal, of the higher indices
    x[3] = torch.linspace(-9, 9, vocab)
    x[4] = torch.linspace(9, -9, vocab)
    x[5] = -INF
    x[6, ::2] = -INF
    x[7, vocab // 3] = NAN
    x[8] = NAN
    x[9, vocab - 1] = INF
    x[10] = torch.finfo(dtype).min
    x[11] = 0.0
    x[11, ::3] = -0.0
    x[12] = x[12].round()                   # many equal ones
    x[13] = 100.0 + 1e-4 * x[13]            # equal in their upper 16 bits
    tokens = torch.randint(0, vocab, (14,), generator=r.g)
    tokens[0], tokens[7] = vocab - 1, vocab // 3
    check_scores(x.to(dtype), tokens, top, pad=1)


# Rows of an odd vocabulary follow each other: every other one begins between two
# words, and its first element is taken by itself.
@pytest.mark.parametrize("vocab", [2049, 2057, 4097, 8199, 33001, 70001])
@pytest.mark.parametrize("dtype,top", [(BF16, 20), (F16, 1), (BF16, 0), (F16, 64)])
def test_scores_of_rows_that_begin_between_words(vocab, dtype, top):
    r = Draw(vocab + top)
    x = r.normal(20, vocab, scale=3.0)
    tokens = torch.randint(0, vocab, (20,), generator=r.g)
    for i in range(2, 20, 2):               # the same in rows of both kinds
        x[i], tokens[i] = x[i + 1], tokens[i + 1] = x[0], 0
    x[2:4, 0] = 30.0                        # the first element is the best
    x[4:6], tokens[4:6] = 0.25, 0           # equal entries
    x[6:8], tokens[6:8] = 0.25, vocab - 1
    x[8:10, 0], tokens[8:10] = NAN, 5
    x[10:12, 0], x[10:12, 1], tokens[10:12] = INF, INF, 1
    x[12:14], tokens[12:14] = -INF, 1
    x[14:16, 1:], tokens[14:16] = -INF, 7   # only the first one is left
    x[16:18], tokens[16:18] = x[16].sort().values, vocab - 1
    x[18:, 0], x[18:, 1], x[18:, 2], tokens[18:] = 9.0, 9.0, 9.0, 1
    check_scores(x.to(dtype), tokens, top)


@pytest.mark.parametrize("vocab,dtype", [(140001, F32), (300007, BF16)])
def test_scores_of_long_rows_in_segments(vocab, dtype):
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(6, vocab, generator=g) * 3
    x[0] = 0.5                              # equal over all segments
    x[1, :] = -INF                          # two entries, in different segments
    x[1, 17] = x[1, vocab - 2] = 1.0
    x[2] = torch.linspace(-20, 20, vocab)   # the best ones all in the last segment
    x[3, vocab // 2] = NAN
    x[4, :vocab // 3] = -INF                # segments without an entry
    x[5] = 0.0
    x[5, 17516:] = 1.0                      # equal ones that begin shortly before a round of reads ends
    tokens = torch.tensor([vocab - 1, vocab - 2, 5, vocab // 2, vocab - 1, 0])
    check_scores(x.to(dtype), tokens, 33)
    check_scores(x.to(dtype), tokens, 0)


def test_the_plain_call_and_the_other_way_are_the_same():
    # a stream of the caller's goes through Python, no stream through the compiled binding
    r = Draw(31)
    here = torch.cuda.current_stream()
    x, w = r.normal(2, 70, 48, dtype=BF16).cuda(), r.normal(48, 4).cuda()
    v = scan_inputs(r, 2, 70, 48, 16, 1, BF16, True, True, True, True, True, True)
    v = {k: cuda(t) for k, t in v.items()}
    _, wd, ws = weights(r, 33, 48)
    ws = ws.cuda()
    logits = r.normal(5, 3000).cuda()
    calls = [
        lambda s: ra.causal_conv(x, w, silu=True, stream=s),
        lambda s: ra.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                                    dt_bias=v["dt_bias"], dt_softplus=True, state=v["state"],
                                    sequence_lens=v["lens"], stream=s),
        lambda s: ra.quantize_rows(x[0, :, :41], stream=s),
        lambda s: [ra.quant_project(x[0], wd, ws, out_dtype=F16, stream=s)],
        lambda s: [ra.quant_project(x.flatten(0, 1), wd, ws, stream=s)],
        lambda s: ra.token_scores(logits, torch.arange(5).cuda(), top=4, stream=s),
        lambda s: ra.token_scores(logits, torch.arange(5, dtype=torch.int32).cuda(), stream=s),
    ]
    for call in calls:
        got, want = call(None), call(here)
        assert type(got) is type(want) and len(got) == len(want)
        for a, b in zip(got, want):
            assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
            assert torch.equal(a, b)
    assert ra.token_scores(logits, top=2).logprob is None
    with pytest.raises(ValueError, match="tap"):
        ra.causal_conv(x, w[:, :0])
    with pytest.raises(ra.RNNError) as e:                # refused by the library in a compiled call
        ra.causal_conv(x, torch.zeros(48, 9).cuda())
    assert e.value.status == ra.RNN_ERR_INVALID_INPUT


@pytest.mark.parametrize("rows,cols,outs", [(1, 8192, 16384), (1, 16000, 8200), (2, 8192, 9000), (4, 4096, 16400),
                                            (16, 1024, 70000), (5, 8000, 9000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_other_types_beside_many_weights(rows, cols, outs, dtype):
    # rounded inside up to 16384 elements, by a launch of its own beyond
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
    w = torch.randint(-127, 128, (outs, cols), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(outs, generator=g, device="cuda") + 0.5
    q = ra.quantize_rows(x)
    total = q.q.double() @ w.double().t().contiguous()          # exact
    y = (total * q.scale.double()[:, None] * ws.double()).cpu().numpy()
    got = ra.quant_project(x, w, ws)
    assert_close(got, y, lm_ref.stored(y, 8 * lm_ref.U * np.abs(y), dtype), "y")
    assert torch.equal(ra.quant_project(q.q, w, ws, x_scale=q.scale, out_dtype=dtype), got)
