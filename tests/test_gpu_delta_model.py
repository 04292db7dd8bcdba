"""The delta-rule example model: its operators together, over a prompt and in beams,
eager and as a captured step."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import delta_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("delta_lm", os.path.join(ROOT, "examples", "delta_lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def model(example):
    return example.Model(layers=2, dim=128, vocab=500, key_heads=2, heads=4, key_dim=32, value_dim=48, seed=3)


def ids(seed, *shape):
    return torch.randint(0, 500, shape, generator=torch.Generator().manual_seed(seed)).cuda()


def test_captured_steps_are_the_eager_ones(example, model):
    prompt = ids(1, 3, 40)
    one, two = (example.Beams(model, prompt, 4, eos=2) for _ in range(2))
    two.capture()
    for _ in range(6):
        one.next()
        torch.cuda.synchronize()
        two.next()
        for a, b in zip(one._moving(), two._moving()):
            assert torch.equal(a, b)


def test_two_captured_searches_side_by_side(example, model):
    """Each graph has its own workspaces: replays on two streams leave both as they are alone."""
    prompts = [ids(5, 2, 30), ids(6, 4, 25)]
    alone = [example.generate(model, p, 6, 3, captured=False) for p in prompts]
    both = [example.Beams(model, p, 3, eos=2) for p in prompts]
    for b in both:
        b.capture()
    streams = [torch.cuda.Stream() for _ in both]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for b, s in zip(both, streams):
            with torch.cuda.stream(s):
                b.next()
    torch.cuda.synchronize()
    for b, (_, scores) in zip(both, alone):
        assert torch.equal(b.scores, scores)


def test_a_beam_is_its_tokens(example, model):
    """After any selections and reorderings a beam's states are those that its tokens
    give when they are fed one at a time, to the bit; and a step's choice is the
    definition's, on the step's own logits."""
    prompt = ids(2, 2, 33)
    search = example.Beams(model, prompt, 3, eos=500 - 1)
    paths = [[[t] for t in row] for row in search.tokens.tolist()]
    for _ in range(5):
        before = search.scores.clone(), search.finished.clone()
        twin = [t.clone() for t in search.state]
        logits = model.logits(model.hidden(search.tokens.view(-1, 1), twin)[:, 0]).view(2, 3, -1)
        search.next()
        _, t, p = delta_ref.beam(logits.cpu(), before[0].cpu(), 3, before[1].cpu(), 499)
        assert np.array_equal(search.tokens.cpu().numpy(), t) and np.array_equal(search.parents.cpu().numpy(), p)
        paths = [[paths[b][i] + [int(tok)] for tok, i in zip(t[b], p[b])] for b in range(2)]
    state = model.new_state(2)
    model.hidden(prompt, state)
    rows = torch.arange(2, device="cuda", dtype=torch.int32)[:, None].expand(2, 3).reshape(1, 6).contiguous()
    state = example.ra.reorder_states(state, rows)
    for i in range(5):
        fed = torch.tensor([path[i] for row in paths for path in row], device="cuda").view(6, 1)
        model.hidden(fed, state)
    for a, b in zip(state, search.state):
        assert torch.equal(a, b)


def test_lengths_are_rows_of_their_own(example, model):
    """A padded batch of prompts, one of them of a single token, is each of them alone."""
    prompt, lens = ids(4, 4, 70), [70, 1, 64, 20]
    state = model.new_state(4)
    x = model.hidden(prompt, state, torch.tensor(lens, dtype=torch.int32).cuda())
    for i, n in enumerate(lens):
        alone = model.new_state(1)
        y = model.hidden(torch.cat([prompt[i:i + 1, :n], prompt[i:i + 1, n:] * 0], 1), alone,
                         torch.tensor([n], dtype=torch.int32).cuda())
        assert torch.equal(x[i, :n], y[0, :n])
        for a, b in zip(state, alone):
            assert torch.equal(a[i], b[0])


def test_generate(example, model):
    prompt = ids(7, 2, 30)
    out, scores = example.generate(model, prompt, 5, beams=4)
    again, same = example.generate(model, prompt, 5, beams=4, captured=False)
    assert out.shape == (2, 4, 5) and scores.shape == (2, 4)
    assert torch.equal(out, again) and torch.equal(scores, same)
    assert (scores < 0).all() and (scores[:, :-1] >= scores[:, 1:]).all()
    for row in out.tolist():                         # no beam twice
        assert len({tuple(beam) for beam in row}) == 4
