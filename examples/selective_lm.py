"""A small selective-state language model on the operators of recurrent_nn_amd.

    python examples/selective_lm.py [--layers 4] [--dim 1024] [--batch 8]
                                    [--prompt 512] [--tokens 64]

Random weights (nothing is downloaded).  A layer norms its tokens, projects
them with 8-bit weights to [x, gate], passes x through the causal convolution,
projects it to step sizes, B and C, runs the selective scan with the gate, and
projects the result back.  The prompt goes through in one call of each
operator; then one token at a time, windows and states replaced in place, in a
captured graph.  The prompt's tokens are scored, and the most likely
alternative is the next token.
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


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.pow(2).mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Linear:
    """A projection with 8-bit weights, one scale for each output."""

    def __init__(self, gen, outs, cols, device, scale=1.0):
        w = torch.randn(outs, cols, generator=gen, device=device) * (scale / math.sqrt(cols))
        self.q, self.scale = ra.quantize_rows(w)

    def __call__(self, x, out_dtype=None):
        y = ra.quant_project(x.flatten(0, -2), self.q, self.scale, out_dtype=out_dtype)
        return y.view(*x.shape[:-1], y.shape[-1])


class Layer:
    def __init__(self, gen, dim, states, taps, device):
        inner, self.low, self.states = 2 * dim, max(16, dim // 16), states

        def uniform(*shape):
            return torch.rand(*shape, generator=gen, device=device)

        self.into = Linear(gen, 2 * inner, dim, device)
        self.taps = (uniform(inner, taps) * 2 - 1) / math.sqrt(taps)
        self.bias = (uniform(inner) * 2 - 1) / math.sqrt(taps)
        self.select = Linear(gen, self.low + 2 * states, inner, device)
        self.step = Linear(gen, inner, self.low, device, scale=0.5)
        size = torch.exp(uniform(inner) * math.log(100.0) + math.log(1e-3))
        self.step_bias = size + torch.log(-torch.expm1(-size))
        self.A = -torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        self.D = torch.ones(inner, device=device)
        self.out = Linear(gen, dim, inner, device, scale=0.5)

    def new_state(self, batch, dtype):
        inner = self.A.shape[0]
        return (torch.zeros(batch, self.taps.shape[1] - 1, inner, device=self.A.device, dtype=dtype),
                torch.zeros(batch, inner, self.states, device=self.A.device))

    def __call__(self, tokens, state, lens=None):
        """tokens [batch, steps, dim]; the window and the state are replaced
        in place."""
        window, h = state
        inner = self.A.shape[0]
        xz = self.into(norm(tokens))
        x, _ = ra.causal_conv(xz[..., :inner], self.taps, self.bias, silu=True, state=window,
                              sequence_lens=lens, state_out=window)
        select = self.select(x)
        low, n = self.low, self.states
        dt = self.step(select[..., :low])
        y, _ = ra.selective_scan(x, dt, self.A, select[..., low:low + n], select[..., low + n:],
                                 D=self.D, z=xz[..., inner:], dt_bias=self.step_bias,
                                 dt_softplus=True, state=h, sequence_lens=lens, state_out=h)
        return tokens + self.out(y)


class Model:
    def __init__(self, layers=4, dim=1024, vocab=32000, states=16, taps=4, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.dtype = dtype
        self.embedding = torch.randn(vocab, dim, generator=gen, device=device).to(dtype)
        self.layers = [Layer(gen, dim, states, taps, device) for _ in range(layers)]
        self.head = Linear(gen, vocab, dim, device, scale=4.0)

    def new_state(self, batch):
        return [layer.new_state(batch, self.dtype) for layer in self.layers]

    def __call__(self, ids, state, lens=None):
        """Logits [batch, steps, vocab] of tokens ids [batch, steps]; the state
        moves on."""
        x = self.embedding[ids]
        for layer, s in zip(self.layers, state):
            x = layer(x, s, lens)
        return self.head(norm(x), out_dtype=torch.float32)


class Decoder:
    """The next tokens of a batch, one step in a captured graph."""

    def __init__(self, model, state, ids):
        self.ids = ids.clone()

        def step():
            logits = model(self.ids[:, None], state)[:, 0]
            best = ra.token_scores(logits, top=1)
            self.ids.copy_(best.top_ids[:, 0])
            self.logprob = best.top_logprobs[:, 0]

        keep = [(w.clone(), h.clone()) for w, h in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            step()
        for (w, h), (w0, h0) in zip(state, keep):       # as before the trial step
            w.copy_(w0)
            h.copy_(h0)
        self.ids.copy_(ids)

    def next(self):
        self.graph.replay()
        return self.ids, self.logprob


def generate(model, prompt, tokens):
    """(score of the prompt's tokens, generated ids [batch, tokens])."""
    state = model.new_state(prompt.shape[0])
    logits = model(prompt, state)
    vocab = logits.shape[-1]
    scores = ra.token_scores(logits[:, :-1].reshape(-1, vocab), prompt[:, 1:].reshape(-1))
    first = ra.token_scores(logits[:, -1], top=1).top_ids[:, 0]
    decoder = Decoder(model, state, first.long())
    out = [first.long()]
    for _ in range(tokens - 1):
        out.append(decoder.next()[0].clone())
    return scores.logprob, torch.stack(out, 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("dim", 1024), ("batch", 8), ("prompt", 512), ("tokens", 64)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    model = Model(layers=a.layers, dim=a.dim)
    prompt = torch.randint(0, 32000, (a.batch, a.prompt), device="cuda")
    generate(model, prompt, 2)                      # kernels and memory warm
    torch.cuda.synchronize()
    t = time.perf_counter()
    logprob, ids = generate(model, prompt, a.tokens)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.batch} x {a.prompt} prompt tokens, mean log probability {logprob.mean().item():.3f}; "
          f"{ids.numel()} tokens generated; {t * 1e3:.1f} ms in all")


if __name__ == "__main__":
    main()
