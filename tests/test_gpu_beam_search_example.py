"""The operators of decoding together, as examples/beam_search.py uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


@pytest.fixture(scope="module")
def example(torch):
    spec = importlib.util.spec_from_file_location("beam_search", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(torch, example):
    model, tokens, scores, ended = example.main(["--requests", "3", "--beams", "4", "--steps", "5", "--hidden", "96",
                                                 "--vocab", "997"])
    assert tokens.shape == (3, 4, 5) and torch.isfinite(scores).all()
    assert (scores[:, :-1] >= scores[:, 1:]).all()                # beams in order of their scores


def test_scores_are_those_of_the_tokens(torch, example):
    """A beam's score is the sum of its tokens' log-probabilities when they are fed one after another:
    states, caches and tokens went to the right beams. The logits agree to the model's FP32 product,
    whose tiles may differ with the rows: 5 steps of at most 1e-3."""
    import fp32_gemm_f32_amd as g
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = example.Model(128, 1009, "cuda", gen)
    state = gen.get_state()
    tokens, scores, ended = example.search(model, 2, 3, 5, 2, gen)
    gen.set_state(state)
    first = torch.randn(2, 1, 128, device="cuda", generator=gen)
    for r in range(2):
        for b in range(3):
            hidden, cache = first[r], torch.zeros(1, 5, 128, device="cuda")
            last, total, over = torch.zeros(1, dtype=torch.int64, device="cuda"), 0.0, False
            for step in range(5):
                hidden = model.advance(hidden, last, cache, step)
                cache[:, step] = hidden
                last = tokens[r, b, step].view(1)
                if not over:
                    total += float(g.token_logprobs(model.head.logits(hidden), last).logprobs)
                over = over or int(last) == 2
            assert abs(total - float(scores[r, b])) < 5e-3, (r, b)
            assert over == bool(ended[r, b])


def test_the_head_is_the_4_bit_one(torch, example):
    gen = torch.Generator(device="cuda").manual_seed(2)
    head = example.Head(torch.randn(301, 95, device="cuda", generator=gen))
    assert head.weight().shape == (301, 95) and head.logits(torch.ones(2, 95, device="cuda")).shape == (2, 301)
