"""A language model's output head in 8 bits: scoring given tokens with alternatives, and one step
of the gradient that training takes back from them.

    python examples/score_tokens.py [--tokens 64] [--hidden 1024] [--vocab 32001] [--top 5]

The head's weights are quantised once. Each call then runs, on the GPU,
    quantize_rows    the hidden states to 8 bits, a scale for each token
    matmul_i8        their product with the weights (both in linear_i8): the logits
    token_logprobs   the given tokens' log-probabilities, entropies and alternatives
    token_logprobs_backward, matmul
                     the gradient of a loss on those, through the logits to the hidden states
Weights and hidden states are random.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp32_gemm_f32_amd as g  # noqa: E402


class Head:
    """An output projection held in 8 bits: (V, K) integers and a scale for each of the V rows."""

    def __init__(self, weight):
        self.q, self.scales = g.quantize_rows(weight)

    def logits(self, hidden):
        return g.linear_i8(hidden, self.q, self.scales)

    def weight(self):
        """The weights the integers stand for, in FP32."""
        return self.q.float() * self.scales[:, None]


def score(head, hidden, tokens, top):
    """(logits, TokenLogprobs) of the tokens that follow the hidden states."""
    logits = head.logits(hidden)
    return logits, g.token_logprobs(logits, tokens, top=top)


def hidden_gradient(head, logits, tokens, scored, entropy_weight):
    """The gradient with respect to the hidden states of
        mean over given tokens of -logprob - entropy_weight * entropy,
    taken through the quantiser as if it were the identity."""
    given = (tokens >= 0).to(torch.float32)
    share = given / given.sum().clamp_min(1)
    d_logits = g.token_logprobs_backward(logits, tokens, scored.lse, scored.entropy, -share,
                                         -entropy_weight * share)
    return g.matmul(d_logits.float(), head.weight())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32001)
    ap.add_argument("--top", type=int, default=5)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    weight = torch.randn(a.vocab, a.hidden, device="cuda", generator=gen) / a.hidden ** 0.5
    hidden = (2 * torch.randn(a.tokens, a.hidden, device="cuda", generator=gen)).to(torch.bfloat16)
    tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=gen)
    tokens[::7] = -100                                  # positions without a token
    head = Head(weight)
    logits, scored = score(head, hidden, tokens, a.top)
    grad = hidden_gradient(head, logits, tokens, scored, 0.01)
    for i in range(min(4, a.tokens)):
        alternatives = ", ".join(f"{t} ({lp:.2f})" for t, lp in zip(scored.top_tokens[i].tolist(),
                                                                    scored.top_logprobs[i].tolist()))
        print(f"token {int(tokens[i]):6d}  logprob {float(scored.logprobs[i]):8.3f}  "
              f"entropy {float(scored.entropy[i]):6.3f}  alternatives {alternatives}")
    print(f"gradient of the hidden states: {tuple(grad.shape)}, norm {float(grad.norm()):.4g}")
    return head, hidden, tokens, logits, scored, grad


if __name__ == "__main__":
    main()
