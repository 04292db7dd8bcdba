"""The sums behind the token scores, to the roundings that their evaluation
makes: rows of two entries, nearly even rows, and rows whose mass lies in one
pack of eight entries anywhere.

U is half a step of float32, relative.  Against a row's maximum M an entry
x = M - g has e = exp2((x - M) log2 e): the difference, the constant and the
product round (3 g U in the exponent), exp2 is one step (2 U).  A reference that
moves multiplies by one more such factor; the distances add up to g, so that it
costs 3 U each time beside.  The hardware's logarithm is taken as one step of
the larger of its result and 1.
"""
import numpy as np
import pytest
import torch

import recurrent_nn_amd as ra
from tests.lm_ref import U
from tests.test_gpu_lm import BF16, F16, F32, INF, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def scores(x, tokens, top=2):
    s = ra.token_scores(x, tokens, top=top)
    return [v.double().cpu().numpy() for v in (s.logprob, s.entropy, s.top_logprobs)]


# ---------------------------------------------------------------------------
# Two entries, 6 to 8 apart, among masked ones
#
# S = 1 + e, e <= 0.0025: one addition rounds (U), e is off by e (3 g + 6) U < 0.1 U,
# the logarithm by 2 U: the log probability of the first one by less than 4 U, which
# is what a row of a model that is nearly certain has to say.  The second one's has
# its difference and the last subtraction beside, U g each.  W = -g e is off by
# g e (3 g + 9) U < 0.5 U.
# ---------------------------------------------------------------------------

PAIRS = [  # vocab, rows, where the first and the second one are
    (2000, 64, 5, 1900), (2000, 64, 1900, 5), (7, 64, 6, 0),
    (6000, 600, 8, 8 + 2048), (6000, 600, 8 + 2048, 8),         # read by one thread
    (6000, 600, 3, 4), (6000, 600, 4, 3),                       # in one load
    (6000, 600, 8, 16 + 2048), (6000, 600, 5000, 8),            # by two threads, two waves
    (6000, 600, 5999, 0), (6000, 600, 0, 5999),
    (6001, 600, 6000, 1), (6001, 600, 0, 2049),
    (200000, 3, 8, 8 + 2048), (200000, 3, 199999, 4), (200000, 3, 100, 150000),   # segments
]


@pytest.mark.parametrize("vocab,rows,first,second", PAIRS)
@pytest.mark.parametrize("masked", ["infinite", "lowest"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_two_entries_apart(vocab, rows, first, second, masked, dtype):
    g = torch.Generator().manual_seed(vocab + first + 3 * second)
    x = torch.full((rows, vocab), -INF if masked == "infinite" else torch.finfo(dtype).min, dtype=dtype)
    top = torch.randn(rows, generator=g) * 3
    x[:, first] = top.to(dtype)
    x[:, second] = (top - 6 - 2 * torch.rand(rows, generator=g)).to(dtype)
    gap = (x[:, first].double() - x[:, second].double()).numpy()
    assert gap.min() > 5.9 and gap.max() < 8.1
    e = np.exp(-gap)
    lse = np.log1p(e)
    x = x.cuda()
    one, h, both = scores(x, torch.full((rows,), first).cuda())
    two, _, _ = scores(x, torch.full((rows,), second).cuda())
    assert np.abs(one + lse).max() <= 4 * U
    assert np.abs(h - (lse + gap * e / (1 + e))).max() <= 4 * U
    assert (np.abs(two + gap + lse) <= (2 * gap + 4) * U).all()
    assert np.array_equal(both, np.stack([one, two], 1))


# ---------------------------------------------------------------------------
# Every entry counts
#
# Sums of a thread: v / 2048 additions of eight entries' (three more deep); W takes
# each entry by itself.  Then 6 over a wave, 4 waves, and up to 9 for segments.  A
# wave's reference moves a dozen times on these rows, and twice at the joins: 16.
# ---------------------------------------------------------------------------

def expected(x):
    """Log probabilities and entropy in 64 bits, and their errors' bounds."""
    x = x.double().cpu().numpy()
    v = x.shape[1]
    d = x - x.max(1, keepdims=True)
    e = np.exp(d)
    S = e.sum(1)
    p, far = e / S[:, None], np.where(e > 0, -d, 0)
    lse = np.log(S)
    moves, joins = 16, 6 + 4 + 9
    rel = (p * (3 * far + 2)).sum(1) + 3 * moves + v / 2048 + 3 + joins
    W = (p * far).sum(1)
    rel_W = (p * far * (3 * far + 4)).sum(1) + W * (5 * moves + v / 256 + joins)
    err = U * (rel + 4 * np.maximum(1, np.abs(lse)))
    err_h = err + U * (rel_W + W * (rel + 2) + lse + W)
    return d - lse[:, None], err, lse + W, err_h


def check(x, tokens):
    logp, err, h, err_h = expected(x)
    got, got_h, _ = scores(x.cuda(), tokens.cuda(), top=0)
    want = logp[np.arange(len(tokens)), tokens.numpy()]
    off = np.abs(got - want) - (err + 2 * U * np.abs(want))
    assert off.max() <= 0, f"log probability: {off.max():.2e} beyond its bound"
    off = np.abs(got_h - h) - err_h
    assert off.max() <= 0, f"entropy: {off.max():.2e} beyond its bound"
    return err


@pytest.mark.parametrize("rows,vocab", [
    (5, 300), (5, 1023), (5, 2048), (513, 2049), (520, 9001), (520, 16390), (3, 131072), (2, 131073),
    (2, 300007), (1, 262144), (64, 40000)])
@pytest.mark.parametrize("scale", [0.05, 3.0])
def test_every_entry_counts(rows, vocab, scale):
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g) * scale
    for dtype in (F32, BF16):
        t = x.to(dtype)
        err = check(t, torch.randint(0, vocab, (rows,), generator=g))
        if scale < 1:                       # the loss of one pack of eight could not hide
            assert err.max() < 8 / vocab * np.exp(-0.5)


@pytest.mark.parametrize("vocab,segmented", [(2049, False), (10247, False), (40961, False), (70001, True)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_mass_in_any_pack(vocab, segmented, dtype):
    # borders of packs, of batches (256 packs a load, two or four loads), of the
    # eight parts of a row and of segments are all multiples of 8 entries
    edges = sorted({min(max(p + s, 0), vocab - 1) // 8 * 8
                    for p in list(range(0, vocab, 2048)) + [vocab - 17, vocab - 8, vocab - 1]
                    for s in (-9, 0, 8)})
    rows = [edges[i:i + 4] for i in range(0, len(edges), 4)] if segmented else [edges]
    for some in rows:                       # (few rows are cut into segments, many are not)
        n = len(some) if segmented else max(len(some), 520)
        x = torch.full((n, vocab), -3.0)
        at = [some[i % len(some)] for i in range(n)]
        for i, p in enumerate(at):
            x[i, p:p + 8] = 12.0 + torch.arange(min(8, vocab - p)) / 8
        check(x.to(dtype), torch.tensor([min(p + i % 8, vocab - 1) for i, p in enumerate(at)]))
