"""Decoding with beam search and an output head in 4 bits.

    python examples/beam_search.py [--requests 4] [--beams 4] [--steps 12] [--hidden 512] [--vocab 32001]

The head's weights are quantised once to microscaled 4-bit floating point. Each step then runs, on the
GPU,
    linear_mx4       the beams' hidden states to 4 bits and their product with the head: the logits
    beam_step        the best continuations of each request's beams, ended beams standing by
    reorder_beams    the caches, the hidden states and the tokens so far, moved to the beams chosen
The model before the head is a stand-in with random weights: a state for each beam, mixed with an
embedding of its last token, and a cache that every step adds a position to.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp32_gemm_f32_amd as g  # noqa: E402


class Head:
    """An output projection held in 4 bits: (V, ceil(K / 2)) bytes and a scale for each 32 elements."""

    def __init__(self, weight):
        self.q, self.scales = g.quantize_mx4(weight)
        self.columns = weight.shape[1]

    def logits(self, hidden):
        return g.linear_mx4(hidden, self.q, self.scales)

    def weight(self):
        """The weights the codes stand for, in FP32."""
        return g.dequantize_mx4(self.q, self.scales, columns=self.columns)


class Model:
    """The stand-in: hidden' = tanh(mix [hidden, embedding of the token, mean of the cache])."""

    def __init__(self, hidden, vocab, device, gen):
        def weight(*shape):
            return torch.randn(*shape, device=device, generator=gen) / shape[-1] ** 0.5
        self.embedding = weight(vocab, hidden)
        self.mix = weight(3 * hidden, hidden)
        self.head = Head(3 * weight(vocab, hidden))

    def advance(self, hidden, tokens, cache, length):
        past = cache[:, :length].mean(dim=1) if length else torch.zeros_like(hidden)
        return torch.tanh(g.matmul(torch.cat([hidden, self.embedding[tokens], past], dim=1), self.mix))


def search(model, requests, beams, steps, eos, gen, device="cuda"):
    """(tokens (requests, beams, steps), scores (requests, beams), beams that have ended) after `steps`
    steps from random states."""
    rows, width = requests * beams, model.mix.shape[1]
    hidden = torch.randn(requests, 1, width, device=device, generator=gen).expand(-1, beams, -1).reshape(rows, width)
    cache = torch.zeros(rows, steps, width, device=device)
    tokens = torch.zeros(rows, steps, dtype=torch.int64, device=device)
    last = torch.zeros(rows, dtype=torch.int64, device=device)
    # all of a request's beams are one at first: only the first counts
    scores = torch.full((requests, beams), -float("inf"), device=device)
    scores[:, 0] = 0
    ended = torch.zeros(requests, beams, dtype=torch.bool, device=device)
    for step in range(steps):
        hidden = model.advance(hidden, last, cache, step)
        cache[:, step] = hidden
        scores, parents, chosen = g.beam_step(model.head.logits(hidden), scores, finished=ended, pad_token=eos)
        live = [hidden, cache[:, :step + 1], tokens[:, :step + 1], ended.view(rows)]
        g.reorder_beams(live, parents, out=live)
        last = chosen.clamp_min(0).view(rows)
        tokens[:, step] = last
        ended |= chosen == eos
    return tokens.view(requests, beams, steps), scores, ended


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=32001)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    model = Model(a.hidden, a.vocab, "cuda", gen)
    tokens, scores, ended = search(model, a.requests, a.beams, a.steps, 2, gen)
    for r in range(min(2, a.requests)):
        for b in range(a.beams):
            print(f"request {r} beam {b}  score {float(scores[r, b]):8.3f}  tokens {tokens[r, b].tolist()}")
    return model, tokens, scores, ended


if __name__ == "__main__":
    main()
