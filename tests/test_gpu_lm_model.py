"""The example model: its operators together, as a prompt, in parts, and
token by token in a captured graph."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(
        "selective_lm", os.path.join(ROOT, "examples", "selective_lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def model(example):
    return example.Model(layers=2, dim=128, vocab=1000, seed=3)


def test_graph_steps_are_the_eager_ones(example, model):
    prompt = torch.randint(0, 1000, (3, 40), generator=torch.Generator().manual_seed(1)).cuda()
    state = model.new_state(3)
    model(prompt, state)
    twin = [(w.clone(), h.clone()) for w, h in state]
    ids = prompt[:, -1].clone()
    decoder = example.Decoder(model, state, ids)
    for _ in range(6):
        best = example.ra.token_scores(model(ids[:, None], twin)[:, 0], top=1)
        ids = best.top_ids[:, 0].long()
        torch.cuda.synchronize()
        got, logprob = decoder.next()
        assert torch.equal(got, ids) and torch.equal(logprob, best.top_logprobs[:, 0])
        for (w, h), (w2, h2) in zip(state, twin):
            assert torch.equal(w, w2) and torch.equal(h, h2)


def test_lengths_are_rows_of_their_own(example, model):
    # rows of a ragged batch end in the state that they reach alone
    g = torch.Generator().manual_seed(2)
    prompt = torch.randint(0, 1000, (4, 33), generator=g).cuda()
    lens = [33, 1, 0, 20]
    state = model.new_state(4)
    model(prompt, state, torch.tensor(lens, dtype=torch.int32).cuda())
    for i, n in enumerate(lens):
        alone = model.new_state(1)
        if n:
            model(prompt[i:i + 1, :n], alone)
        # the first layer has the same inputs: the window to the bit, the state
        # as far as two orders of float32 operations may part (33 steps, each off
        # by at most 40 half steps of float32: 8e-5)
        assert torch.equal(state[0][0][i], alone[0][0][0])
        scale = alone[0][1].abs().max().clamp(min=1e-6)
        assert ((state[0][1][i] - alone[0][1][0]).abs().max() / scale) < 1e-4
        if n == 0:
            for w, h in state:
                assert not w[i].any() and not h[i].any()


def test_generate(example, model):
    prompt = torch.randint(0, 1000, (2, 30), generator=torch.Generator().manual_seed(4)).cuda()
    logprob, ids = example.generate(model, prompt, 5)
    again, same = example.generate(model, prompt, 5)
    assert logprob.shape == (58,) and ids.shape == (2, 5)
    assert torch.isfinite(logprob).all() and (logprob < 0).all()
    assert torch.equal(logprob, again) and torch.equal(ids, same)
