"""The example that runs the quantiser, the 8-bit product, the log-probabilities, their gradient
and the FP32 product together, against the formulas in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example(capsys):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("score_tokens", os.path.join(ROOT, "examples", "score_tokens.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    T, K, V, top = 33, 200, 1003, 3
    head, hidden, tokens, logits, scored, grad = example.main(
        ["--tokens", str(T), "--hidden", str(K), "--vocab", str(V), "--top", str(top)])
    assert "gradient of the hidden states" in capsys.readouterr().out
    w = head.weight().double().cpu().numpy()
    h = hidden.double().cpu().numpy()
    x = logits.double().cpu().numpy()
    tok = tokens.cpu().numpy()

    # logits: hidden states off by half a step of their scale each, then one rounding to bf16
    step = np.abs(h).max(1, keepdims=True) / 254 * (1 + 2.0 ** -10)
    want = h @ w.T
    bound = step * np.abs(w).sum(1)[None, :] + 2.0 ** -8 * np.abs(x) + 1e-5
    assert (np.abs(x - want) <= bound).all()

    # log-probabilities and alternatives of the logits as they are
    m = x.max(1, keepdims=True)
    lse = (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]
    lp = np.where(tok < 0, 0.0, x[np.arange(T), np.maximum(tok, 0)] - lse)
    p = np.exp(x - lse[:, None])
    ent = -(p * (x - lse[:, None])).sum(1)
    close = dict(rtol=0, atol=(64 + V / 256 + 32) * 2.0 ** -23 * (2 * np.log(V) + 2))
    np.testing.assert_allclose(scored.logprobs.double().cpu().numpy(), lp, **close)
    np.testing.assert_allclose(scored.entropy.double().cpu().numpy(), ent, **close)
    order = np.stack([np.lexsort((np.arange(V), -x[i]))[:top] for i in range(T)])
    assert np.array_equal(scored.top_tokens.cpu().numpy(), order)

    # the gradient: half a step of bf16 on each gradient of a logit, and FP32's sum over V
    share = (tok >= 0) / (tok >= 0).sum()
    hot = np.zeros_like(x)
    hot[np.arange(T)[tok >= 0], tok[tok >= 0]] = 1
    d = -share[:, None] * (hot - p) + 0.01 * share[:, None] * p * (x - lse[:, None] + ent[:, None])
    off = np.abs(d) * (2.0 ** -8 + 2.0 ** -16)
    tol = off @ np.abs(w) + (np.abs(d) @ np.abs(w)) * (V + 8) * 2.0 ** -24 + 1e-12
    assert (np.abs(grad.double().cpu().numpy() - d @ w) <= tol).all()
