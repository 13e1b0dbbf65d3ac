"""The beam step's log-sum-exp for logits far from 0, against 64 bits."""
import math

import pytest

import fp32_gemm_f32_amd as g
from test_gpu_gemm_i8 import dtype_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def check(torch, x, what=None):
    """With one beam and a score of 0 the best continuation's total is peak - log-sum-exp = -log(sum of
    e^(x - peak)). A thread adds 128 terms at most: rows under 16384 by 256 threads, 64 of them; longer
    ones in parts of 8192, or 512 and 1024 threads, 128 up to 131072. Half a step (2^-24) for each addition, 24
    for the joins of lanes and waves, 2 for an exponential, log2 V <= 17 for arguments and the
    constant, whose errors are relative to a term's distance from the peak, and the result's own."""
    want = what if what is not None else -(x.double() - x.double().amax(1, keepdim=True)).exp().sum(1).log()
    got = g.beam_step(x, torch.zeros(len(x), 1, device="cuda")).scores[:, 0].double()
    bound = (128 + 24 + 2 + 17 + want.abs()) * 2.0 ** -24
    worst = ((got - want).abs() / bound).max()
    assert worst <= 1, (float(worst), got[:4], want[:4])
    return got - want


AT = [0.0, 9.3, 30.0, -100.0, 301.7, 1000.0, -5000.0, 60000.0]
SHAPES = [(1, 2000), (4, 16001), (3, 131072), (300, 5003), (300, 70008)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("at", AT)
def test_logits_around_a_number(torch, dtype, rows, V, at):
    """All alike, the case in which every thread has the same peak; few distinct ones; and normal ones."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    t = dtype_of(torch, dtype)
    print(f"[beam sums] {dtype} {rows}x{V} at {at}", flush=True)
    check(torch, torch.full((rows, V), at, device="cuda").to(t))
    few = torch.randint(-2, 3, (rows, V), device="cuda", generator=gen)
    check(torch, (at + few).to(t))
    check(torch, (at + 2 * torch.randn(rows, V, device="cuda", generator=gen)).to(t))


@pytest.mark.parametrize("at", [30.0, 301.7, 1000.0, -5000.0])
def test_a_shift_moves_no_total(torch, at):
    """Beams whose rows differ by a constant alone: multiples of 2^-6, so that the shifted logits are exact.
    Their order is that of the scores, which differ by four times what the sums of 2000 terms may be off
    (8 terms to a thread) and far less than two logits: first come the largest logit's tokens of every beam."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    base = torch.randint(-200, 200, (1, 2000), device="cuda", generator=gen).float() / 64
    at = math.floor(at * 64) / 64
    shifts = torch.tensor([0.0, at, at / 2, -at], device="cuda")
    gap = 4 * (8 + 24 + 2 + 11) * 2.0 ** -24
    order = torch.tensor([2, 0, 3, 1], device="cuda")
    scores = torch.empty(1, 4, device="cuda")
    scores[0, order] = -gap * torch.arange(4, device="cuda", dtype=torch.float32)
    best = (base[0] == base.max()).nonzero()[:, 0]
    assert 4 * len(best) <= 64
    r = g.beam_step(base + (shifts * 64).round()[:, None] / 64, scores, top=4 * len(best))
    assert torch.equal(r.beams[0], order.repeat_interleave(len(best)))
    assert torch.equal(r.tokens[0], best.repeat(4))
