"""A small delta-rule language model on the operators of recurrent_nn_amd, decoded
with several beams.

    python examples/delta_lm.py [--layers 4] [--dim 1024] [--batch 8] [--beams 4]
                                [--prompt 512] [--tokens 64]

Random weights (nothing is downloaded).  A layer norms its tokens, projects them
with 8-bit weights to [queries, keys, values, gate, rates, decays], passes the
first three through the causal convolution, runs the gated delta rule, norms each
head's outputs with the gate, and projects the result back.  The prompts go
through in one call of each operator; their windows and states are then copied to
the beams of each request, and one token at a time, in a captured graph, the beams
move on: the best continuations are selected and the states put in their order.
"""
import argparse
import math
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import recurrent_nn_amd as ra  # noqa: E402


class Linear:
    """A projection with 8-bit weights, one scale for each output."""

    def __init__(self, gen, outs, cols, device, scale=1.0):
        w = torch.randn(outs, cols, generator=gen, device=device) * (scale / math.sqrt(cols))
        self.q, self.scale = ra.quantize_rows(w)

    def __call__(self, x, out_dtype=None):
        y = ra.quant_project(x.flatten(0, -2), self.q, self.scale, out_dtype=out_dtype)
        return y.view(*x.shape[:-1], y.shape[-1])


class Norm:
    def __init__(self, dim, device):
        self.weight = torch.ones(dim, device=device)

    def __call__(self, x):
        return ra.gated_norm(x.flatten(0, -2), self.weight).view(x.shape)


class Layer:
    def __init__(self, gen, dim, key_heads, heads, key_dim, value_dim, taps, device):
        self.key_heads, self.heads, self.key_dim, self.value_dim = key_heads, heads, key_dim, value_dim
        keys, values = key_heads * key_dim, heads * value_dim
        self.sizes = [2 * keys + values, values, heads, heads]

        def uniform(*shape):
            return torch.rand(*shape, generator=gen, device=device)

        self.norm = Norm(dim, device)
        self.into = Linear(gen, sum(self.sizes), dim, device)
        self.taps = (uniform(self.sizes[0], taps) * 2 - 1) / math.sqrt(taps)
        size = torch.exp(uniform(heads) * math.log(100.0) + math.log(1e-3))
        self.step_bias = size + torch.log(-torch.expm1(-size))
        self.A = -(1 + 15 * uniform(heads))
        self.weight = torch.ones(value_dim, device=device)
        self.out = Linear(gen, dim, values, device, scale=0.5)

    def new_state(self, batch, dtype):
        return [torch.zeros(batch, self.taps.shape[1] - 1, self.taps.shape[0], device=self.A.device, dtype=dtype),
                torch.zeros(batch, self.heads, self.key_dim, self.value_dim, device=self.A.device)]

    def __call__(self, tokens, state, lens=None):
        """tokens [batch, steps, dim]; the window and the state are replaced in
        place."""
        window, S = state
        x, z, rate, decay = self.into(self.norm(tokens)).split(self.sizes, 2)
        x, _ = ra.causal_conv(x, self.taps, silu=True, state=window, sequence_lens=lens, state_out=window)
        keys = self.key_heads * self.key_dim
        q, k = (x[..., i * keys:(i + 1) * keys].unflatten(2, (self.key_heads, self.key_dim)) for i in (0, 1))
        v = x[..., 2 * keys:].unflatten(2, (self.heads, self.value_dim))
        o, _ = ra.gated_delta(q, k, v, rate, g=decay, A=self.A, dt_bias=self.step_bias, beta_sigmoid=True,
                              normalize=True, state=S, sequence_lens=lens, state_out=S)
        rows = tokens.shape[0] * tokens.shape[1]
        o = o.view(rows, self.heads, self.value_dim)
        z = z.flatten(0, 1).unflatten(1, (self.heads, self.value_dim))
        y = ra.gated_norm(o, self.weight, z=z, out=o)
        return tokens + self.out(y.view(*tokens.shape[:2], -1))


class Model:
    def __init__(self, layers=4, dim=1024, vocab=32000, key_heads=4, heads=8, key_dim=128, value_dim=128, taps=4,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.dtype, self.vocab = dtype, vocab
        self.embedding = torch.randn(vocab, dim, generator=gen, device=device).to(dtype)
        self.layers = [Layer(gen, dim, key_heads, heads, key_dim, value_dim, taps, device) for _ in range(layers)]
        self.norm = Norm(dim, device)
        self.head = Linear(gen, vocab, dim, device, scale=4.0)

    def new_state(self, batch):
        return [t for layer in self.layers for t in layer.new_state(batch, self.dtype)]

    def hidden(self, ids, state, lens=None):
        """Rows [batch, steps, dim] of tokens ids [batch, steps]; the state moves on."""
        x = self.embedding[ids]
        for i, layer in enumerate(self.layers):
            x = layer(x, state[2 * i:2 * i + 2], lens)
        return x

    def logits(self, x):
        return self.head(self.norm(x), out_dtype=torch.float32)


class Beams:
    """The beams of a batch of prompts [batch, steps], one step in a captured graph."""

    def __init__(self, model, prompt, beams, eos, lens=None):
        self.model, self.eos = model, eos
        batch, steps = prompt.shape
        state = model.new_state(batch)
        x = model.hidden(prompt, state, lens)
        last = x[:, -1] if lens is None else x[torch.arange(batch, device=x.device), lens.long().clamp(min=1) - 1]
        first = ra.beam_select(model.logits(last)[:, None], torch.zeros(batch, 1, device=x.device), keep=beams)
        self.state = ra.reorder_states(state, first.parents)
        self.scores, self.finished = first.scores, first.tokens == eos
        self.tokens, self.parents = first.tokens, first.parents
        self.graph = None

    def step(self):
        ids = self.tokens.clamp(min=0).view(-1, 1)
        logits = self.model.logits(self.model.hidden(ids, self.state)[:, 0])
        best = ra.beam_select(logits.view(*self.tokens.shape, -1), self.scores, finished=self.finished, eos=self.eos)
        ra.reorder_states(self.state, best.parents, out=self.state)
        self.scores.copy_(best.scores)
        self.finished.copy_(best.tokens == self.eos)
        self.tokens.copy_(best.tokens)
        self.parents.copy_(best.parents)

    def capture(self):
        kept = [t.clone() for t in self._moving()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        for t, was in zip(self._moving(), kept):        # as before the trial step
            t.copy_(was)

    def _moving(self):
        return [*self.state, self.scores, self.finished, self.tokens, self.parents]

    def next(self):
        if self.graph is None:
            self.step()
        else:
            self.graph.replay()


def generate(model, prompt, tokens, beams=4, eos=2, lens=None, captured=True):
    """(ids [batch, beams, tokens], best first; their sums of log probabilities)."""
    search = Beams(model, prompt, beams, eos, lens)
    if captured:
        search.capture()
    trace = [(search.tokens.clone(), search.parents.clone())]
    for _ in range(tokens - 1):
        search.next()
        trace.append((search.tokens.clone(), search.parents.clone()))
    # back from each last token along its parents
    at = torch.arange(beams, device=prompt.device).expand(prompt.shape[0], beams)
    out = []
    for ids, parents in reversed(trace):
        out.append(ids.gather(1, at))
        at = parents.long().clamp(min=0).gather(1, at)
    return torch.stack(out[::-1], 2), search.scores


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("dim", 1024), ("batch", 8), ("beams", 4), ("prompt", 512), ("tokens", 64)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    model = Model(layers=a.layers, dim=a.dim)
    prompt = torch.randint(0, model.vocab, (a.batch, a.prompt), device="cuda")
    generate(model, prompt, 2, a.beams)             # kernels and memory warm
    torch.cuda.synchronize()
    t = time.perf_counter()
    ids, scores = generate(model, prompt, a.tokens, a.beams)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.batch} x {a.prompt} prompt tokens, {a.tokens} tokens in {a.beams} beams each, mean log probability "
          f"of the best {scores[:, 0].mean().item() / a.tokens:.3f}; {t * 1e3:.1f} ms in all")


if __name__ == "__main__":
    main()
