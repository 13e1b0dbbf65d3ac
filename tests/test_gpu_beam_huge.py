"""The beam step for logits of any size, against 64 bits: rows around numbers whose FP32 neighbours lie far
apart, and masks of such numbers."""
import pytest

import fp32_gemm_f32_amd as g
from test_gpu_beam_sums import check, torch  # noqa: F401  (a fixture)
from test_gpu_gemm_i8 import dtype_of

pytestmark = pytest.mark.gpu

AT = [1e8, 9.9e8, 1.4e9, -2e9, 5e9, 1e10, -1e10, 1e15, -1e20, 1e29, 5e29, -2e30, 3e38, -3.3e38]
SHAPES = [(2, 7), (3, 2000), (2, 40000), (300, 70008)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", AT)
def test_rows_around_a_huge_number(torch, dtype, rows, V, at):
    """All alike, and neighbours of the type: e^-(their distance) is 0 or nearly so."""
    t = dtype_of(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.full((rows, V), at, device="cuda").to(t)
    print(f"[huge] {dtype} {rows}x{V} at {at}", flush=True)
    check(torch, x)
    for few in (0.5, 0.001):
        if dtype == "f32":
            lower = torch.nextafter(x, torch.tensor(-3.4e38, device="cuda"))
        else:
            lower = x * (1 + 2 ** -7 * (-1 if at > 0 else 1))
        y = torch.where(torch.rand(rows, V, device="cuda", generator=gen) < few, x, lower.to(t))
        assert torch.isfinite(y.float()).all()
        check(torch, y)


@pytest.mark.parametrize("V", [300, 2000, 40000])
def test_where_neighbours_are_64_apart(torch, V):
    """Peaks on both sides of 2^30, beyond which the sums' reference is taken in another way, in any order of
    threads, waves and parts."""
    a = 2.0 ** 30
    gen = torch.Generator(device="cuda").manual_seed(V)
    for sign in (1, -1):
        values = sign * torch.tensor([a - 128, a - 64, a, a + 128, a + 256], device="cuda")
        for n in (2, 3, 4, 5):
            for first in range(0, 6 - n):
                x = values[first:first + n][torch.randint(0, n, (5, V), device="cuda", generator=gen)]
                check(torch, x)
                check(torch, x.sort(dim=1).values)
                check(torch, x.sort(dim=1, descending=True).values)


@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e30, -3.0e38])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_tokens_and_beams(torch, dtype, mask):
    """Banned tokens hold a huge negative number; of a beam with nothing else all are alike."""
    t = dtype_of(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(3)
    V = 5000
    x = torch.randn(8, V, device="cuda", generator=gen)
    x[:, torch.rand(V, device="cuda", generator=gen) < 0.5] = mask
    x[3] = mask
    x[5, 1:] = mask
    x = x.to(t)
    check(torch, x)
    scores = torch.tensor([[-1.0, -2.0, -1.5, -0.5, -1.0, -30.0, -2.0, -1.0]], device="cuda")
    r = g.beam_step(x, scores, top=8)
    total = x.double() - x.double().amax(1, keepdim=True)
    total = total - total.exp().sum(1, keepdim=True).log() + scores.double().T
    want = total.flatten().sort(descending=True, stable=True)
    assert ((r.scores[0].double() - want.values[:8]).abs() <= 200 * 2.0 ** -24 + 2.0 ** -24 * want.values[:8].abs()).all()
    # (the masked beam's tokens are alike, each with log(1 / V): none of the first eight)
    assert torch.equal(r.beams[0], want.indices[:8] // V) and torch.equal(r.tokens[0], want.indices[:8] % V)
