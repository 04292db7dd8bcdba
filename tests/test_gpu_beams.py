"""Gated norm, beam selection and reordering of states on the GPU against their
plain definitions (tests/delta_ref.py): whole numbers exactly, sums within
bounds that count roundings."""
import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from tests import delta_ref
from tests.lm_ref import U, assert_close
from tests.test_gpu_lm import BF16, F16, F32, INF, NAN, Draw, cuda, inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ra._lib.load()
    yield


# ---------------------------------------------------------------------------
# Gated norm
# ---------------------------------------------------------------------------

NORM = [  # rows, groups, dim, dtype, gate, shared weight, pad
    (1, 1, 1, F32, None, True, 0), (3, 1, 7, BF16, "after", True, 1), (5, 3, 32, F16, "before", False, 0),
    (64, 4, 128, BF16, "after", True, 8), (2, 5, 33, F32, "after", False, 3), (7, 2, 64, BF16, None, True, 0),
    (9, 3, 256, F16, "after", True, 0), (4, 2, 257, F32, "before", True, 5), (3, 1, 1000, BF16, "after", True, 24),
    (2, 1, 2048, F32, "after", True, 0), (2, 2, 2049, F16, None, False, 1), (3, 1, 5001, BF16, "before", True, 7),
    (2, 1, 8192, F32, "after", True, 0), (2, 1, 9001, F16, "after", True, 0), (1, 1, 40000, F32, "before", True, 0),
    (1, 2, 70001, BF16, "after", False, 1), (1000, 1, 16, F32, "after", True, 0),
    (33, 3, 40, BF16, "after", True, 0), (65, 1, 63, F16, "before", True, 1), (9, 7, 72, F32, "after", False, 0),
    (350, 3, 600, BF16, "after", True, 0), (513, 2, 1023, F16, "before", True, 1), (3, 2, 1024, F32, None, True, 0),
    (1024, 1, 513, BF16, "after", True, 3), (2, 1, 1500, BF16, "after", True, 0), (2, 1, 3001, F32, "before", True, 1),
    (3, 1, 4096, F16, "after", True, 0), (2, 1, 4097, BF16, "after", True, 0), (1, 1, 16384, BF16, None, True, 0),
]


@pytest.mark.parametrize("k", range(len(NORM)))
def test_norm(k):
    rows, groups, dim, dtype, gate, shared, pad = NORM[k]
    r = Draw(700 + k)
    x = r.normal(rows, groups, dim, dtype=dtype, scale=2.0)
    w = r.normal(dim) if shared else r.normal(groups, dim)
    z = r.normal(rows, groups, dim, dtype=dtype, scale=3.0) if gate else None
    y, err = delta_ref.norm(x, w, z, gate == "before", 1e-6)
    xd, zd = inside(x, pad), inside(z, pad) if gate else None
    got = ra.gated_norm(xd, cuda(w), z=zd, gate_first=gate == "before")
    assert got.dtype == dtype
    assert_close(got, y, err, "y")
    out = inside(torch.zeros_like(x), 5)
    ra.gated_norm(xd, cuda(w), z=zd, gate_first=gate == "before", out=out, stream=torch.cuda.current_stream())
    assert torch.equal(out, got)
    for place in (xd, zd):                              # in place of either
        if place is not None:
            was = place.clone()
            assert ra.gated_norm(xd, cuda(w), z=zd, gate_first=gate == "before", out=place) is not None
            assert torch.equal(place, got)
            place.copy_(was)
    if groups == 1:                                     # rows of two dimensions
        flat = ra.gated_norm(xd[:, 0], cuda(w).view(dim), z=zd[:, 0] if gate else None, gate_first=gate == "before")
        assert torch.equal(flat, got[:, 0])


def test_norm_edges():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    assert not ra.gated_norm(x, w).any()                                # zeros over sqrt(eps)
    assert ra.gated_norm(x, w, eps=0.0).isnan().all()                   # 0 / 0, as the formula says
    x[1], x[2, 5], x[3] = 1e30, NAN, 3.0
    y = ra.gated_norm(x, w)
    assert not y[1].any()                                               # the sum of squares is beyond float32
    assert y[2].isnan().all() and torch.allclose(y[3], torch.ones(64, device="cuda"), rtol=1e-6, atol=0)
    z = torch.full((4, 64), -200.0, device="cuda")
    assert not ra.gated_norm(x[3:], w, z=z[3:])[0].abs().gt(1e-30).any()
    for empty in ((0, 2, 8), (2, 0, 8), (2, 2, 0)):
        assert ra.gated_norm(torch.empty(empty, device="cuda"), torch.ones(empty[2], device="cuda")).shape == empty


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------

BEAM = [  # batch, beams, vocab, keep, dtype, finished, masked, pad
    (1, 1, 1, 1, F32, False, False, 0), (2, 3, 5, 4, BF16, True, True, 1), (3, 4, 100, 8, F16, True, False, 0),
    (2, 2, 7, 16, F32, False, True, 0), (4, 8, 1000, 8, BF16, False, False, 0), (1, 4, 2049, 8, F32, True, True, 3),
    (2, 5, 4097, 5, BF16, False, True, 1), (1, 64, 300, 64, F32, True, False, 0), (3, 16, 9001, 32, F16, True, True, 1),
    (1, 1, 50000, 64, BF16, False, False, 0), (1, 4, 100001, 8, F32, True, True, 0), (2, 3, 70003, 6, BF16, False, False, 5),
    (1, 64, 20000, 64, BF16, False, False, 0), (200, 4, 600, 4, BF16, True, False, 0),
]


def beam_case(k):
    b, n, v, keep, dtype, finished, masked, pad = BEAM[k]
    r = Draw(800 + k)
    x = r.normal(b, n, v, scale=2.5)
    if masked:
        x[r.uniform(b, n, v) < 0.5] = -INF
    x = x.to(dtype)
    scores = -20 * r.uniform(b, 1) - 2 * r.uniform(b, n)
    ended = r.uniform(b, n) < 0.4 if finished else None
    return x, scores, ended, keep, pad


def check_beam(got, x, scores, keep, ended=None, eos=0):
    s, t, p = delta_ref.beam(x, scores, keep, ended, eos)
    assert got.scores.dtype == F32 and got.tokens.dtype == torch.int32 and got.parents.dtype == torch.int32
    assert np.array_equal(got.parents.cpu().numpy(), p) and np.array_equal(got.tokens.cpu().numpy(), t)
    # the normaliser: exponentials of 2 to 3 roundings, summed in 64 bits by eights
    # (3 more), and the value's own rounding
    top = max(1.0, x.float().nan_to_num(0, 0, 0).abs().max().item())
    assert_close(got.scores, s, 2 * U * (8 + 2 * top) + np.abs(np.nan_to_num(s, posinf=0, neginf=0)) * U, "scores")


@pytest.mark.parametrize("k", range(len(BEAM)))
def test_beam(k):
    x, scores, ended, keep, pad = beam_case(k)
    eos = x.shape[2] // 2
    more = dict(finished=cuda(ended), eos=eos) if ended is not None else {}
    xd = inside(x, pad)
    got = ra.beam_select(xd, cuda(scores), keep=keep, **more)
    check_beam(got, x, scores, keep, ended, eos)
    again = ra.beam_select(xd, cuda(scores), keep=keep, **more, stream=torch.cuda.current_stream())
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,vocab", [(F32, 999), (BF16, 999), (BF16, 40001), (F16, 70001)])
def test_equal_beams_keep_their_order(dtype, vocab):
    """Rows with the same entries at unlike alignments, and equal entries: ties
    go by beam, then by token."""
    r = Draw(21)
    row = r.normal(vocab, scale=2.0).to(dtype)
    x = row.repeat(2, 6, 1)
    scores = torch.full((2, 6), -3.0)
    scores[1, 2:] = -1.0
    check_beam(ra.beam_select(x.cuda(), scores.cuda(), keep=12), x, scores, 12)
    x = torch.zeros(1, 3, vocab, dtype=dtype)           # every entry equal
    scores = torch.tensor([[-1.0, -1.0, -0.5]])
    check_beam(ra.beam_select(x.cuda(), scores.cuda(), keep=64), x, scores, 64)
    x[0, 2] = -INF
    x[0, 2, vocab - 3:] = 1.0                           # a few entries in one beam
    check_beam(ra.beam_select(x.cuda(), scores.cuda(), keep=7), x, scores, 7)


def test_beams_without_candidates():
    r = Draw(22)
    x = r.normal(6, 3, 500)
    scores = -r.uniform(6, 3)
    ended = torch.zeros(6, 3, dtype=torch.bool)
    x[0] = -INF                                         # nothing allowed
    x[1, 0, 5], x[1, 1, 7] = NAN, INF                   # two beams without a distribution
    scores[2] = -INF                                    # no beam at all
    scores[3, 1:] = -INF                                # the first step
    scores[3, 2] = NAN
    ended[4] = True                                     # all finished
    ended[5, 1] = True
    scores[5, 1] = -INF                                 # finished and not there
    x[4, 0] = NAN                                       # (a finished beam's logits are not read)
    for keep in (1, 3, 9):
        got = ra.beam_select(x.cuda(), scores.cuda(), keep=keep, finished=ended.cuda(), eos=4)
        check_beam(got, x, scores, keep, ended, 4)
        byte = ra.beam_select(x.cuda(), scores.cuda(), keep=keep, finished=ended.byte().cuda(), eos=4)
        for a, b in zip(got, byte):
            assert torch.equal(a, b)


def test_few_entries_among_masked_ones():
    """-inf but for one entry here and there, in long rows cut into segments."""
    x = torch.full((1, 2, 90001), -INF)
    x[0, 0, 90000], x[0, 1, 0], x[0, 1, 45000] = 2.0, -50.0, -50.0
    scores = torch.tensor([[-4.0, -3.9]])
    check_beam(ra.beam_select(x.cuda(), scores.cuda(), keep=6), x, scores, 6)


def test_rising_and_falling_rows():
    v = 30000
    up = torch.linspace(-30, 30, v)
    x = torch.stack([up, up.flip(0), up * 3, -up.abs()])[None]
    scores = torch.tensor([[-1.0, -1.5, -0.2, -0.1]])
    check_beam(ra.beam_select(x.cuda(), scores.cuda(), keep=16), x, scores, 16)


def test_beam_in_a_graph():
    x, scores, ended, keep, _ = beam_case(10)
    xd, sd, ed = x.cuda(), scores.cuda(), ended.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ra.beam_select(xd, sd, keep=keep, finished=ed, eos=3)
    for k in range(4):
        sd.copy_(scores + 0.1 * k * torch.arange(scores.shape[1]))
        ed.copy_(ended ^ bool(k % 2))
        graph.replay()
        torch.cuda.synchronize()
        want = ra.beam_select(xd, sd, keep=keep, finished=ed, eos=3)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert ra.beam_select(xd[:0], sd[:0], keep=2).tokens.shape == (0, 2)


# ---------------------------------------------------------------------------
# Reordering
# ---------------------------------------------------------------------------

def states_of(r, rows):
    return [(r.normal(rows, 3, 40, dtype=BF16), 0), (r.normal(rows, 2, 8, 8), 0), (r.normal(2, rows, 65), 1),
            ((r.uniform(rows, 7) * 100).to(torch.int8), 0), (r.normal(rows, dtype=F16), 0),
            (r.normal(2, 3, rows, 5, dtype=torch.float64), 2), (torch.empty(rows, 0), 0),
            (r.uniform(rows, 33) < 0.5, 0), (r.normal(rows, 4096), 0)]


@pytest.mark.parametrize("batch,beams,keep", [(1, 1, 1), (3, 4, 4), (2, 5, 5), (4, 1, 6), (2, 8, 3), (1, 17, 17),
                                              (2, 33, 33), (1, 64, 64), (2, 3, 80), (1, 100, 20)])
def test_reorder(batch, beams, keep):
    r = Draw(900 + beams)
    states = states_of(r, batch * beams)
    parents = torch.randint(0, beams, (batch, keep), generator=r.g, dtype=torch.int32)
    dims = [n for _, n in states]
    dev = [s.cuda() for s, _ in states]
    want = [delta_ref.reorder(s, parents, n) for s, n in states]
    got = ra.reorder_states(dev, parents.cuda(), dim=dims)
    for g, w, (s, _) in zip(got, want, states):
        assert g.dtype == s.dtype and torch.equal(g.cpu(), w)
    zero = [i for i, n in enumerate(dims) if n == 0]            # the compiled call
    fast = ra.reorder_states([dev[i] for i in zero], parents.cuda())
    for i, g in zip(zero, fast):
        assert torch.equal(g.cpu(), want[i])
    out = [torch.zeros_like(g) for g in got]
    ra.reorder_states(dev, parents.cuda(), dim=dims, out=out, stream=torch.cuda.current_stream())
    for o, w in zip(out, want):
        assert torch.equal(o.cpu(), w)
    if keep == beams and beams <= 64:                           # in place
        hold = ra.reorder_states(dev, parents.cuda(), dim=dims, out=dev)
        for h, s, w in zip(hold, dev, want):
            assert h is s and torch.equal(s.cpu(), w)


def test_reorder_many_tensors_and_odd_places():
    """More tensors than a launch takes, at addresses of every alignment."""
    r = Draw(31)
    parents = torch.randint(0, 4, (3, 4), generator=r.g, dtype=torch.int32)
    flat = (r.uniform(80, 12 * 61 + 80) * 200).to(torch.uint8).cuda()
    dev = [flat[i, i:i + 12 * 61].view(12, 61) for i in range(80)]
    want = [delta_ref.reorder(s.cpu(), parents, 0) for s in dev]
    for g, w in zip(ra.reorder_states(dev, parents.cuda()), want):
        assert torch.equal(g.cpu(), w)
    before = flat.clone()
    ra.reorder_states(dev, parents.cuda(), out=dev)
    for i, w in enumerate(want):
        assert torch.equal(dev[i].cpu(), w)
        assert torch.equal(flat[i, :i], before[i, :i]) and torch.equal(flat[i, i + 732:], before[i, i + 732:])


def test_parents_beyond_their_range_are_bounded():
    r = Draw(32)
    x = r.normal(6, 40).cuda()
    parents = torch.tensor([[-3, 7, 1], [2147483647, -2147483648, 2]], dtype=torch.int32)
    got, = ra.reorder_states([x], parents.cuda())
    assert torch.equal(got.cpu(), delta_ref.reorder(x.cpu(), parents, 0))
    ra.reorder_states([x], parents.cuda(), out=[x])
    assert torch.equal(got, x)


def test_reorder_in_a_graph_and_nothing_to_do():
    r = Draw(33)
    x, y = r.normal(8, 1000).cuda(), r.normal(2, 8, 24, dtype=BF16).cuda()
    parents = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.reorder_states([x, y], parents, dim=[0, 1], out=[x, y])
    for k in range(4):
        parents.copy_(torch.randint(0, 4, (2, 4), generator=r.g, dtype=torch.int32))
        x.copy_(r.normal(8, 1000))
        want = [delta_ref.reorder(s.cpu(), parents.cpu(), n) for s, n in ((x, 0), (y, 1))]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.cpu(), want[0]) and torch.equal(y.cpu(), want[1])
    assert ra.reorder_states([], parents) == []
    assert ra.reorder_states([x[:0]], parents[:0])[0].shape == (0, 1000)
    assert ra.reorder_states([x], parents[:, :0])[0].shape == (0, 1000)
