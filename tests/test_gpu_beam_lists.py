"""The selection of a beam's best logits from long rows, whose threads hold more of them than their
registers: best ones alone in their threads, several to a thread, and both in one row; few distinct
values, whose equal ones overflow the list of candidates."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g
from test_gpu_gemm_i8 import dtype_of

pytestmark = pytest.mark.gpu

ROWS = 300                                        # more than compute units: rows are not split
THREADS = 1024


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def step(torch, x, top):
    """One beam to a request: continuations in the order of its logits, equal ones by their tokens."""
    r = g.beam_step(x, torch.zeros(len(x), 1, device="cuda"), top=top)
    assert (r.beams == 0).all()
    return r


@pytest.mark.parametrize("V", [70008, 131072, 90001])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_best_ones_alone_and_together(torch, dtype, V):
    """24 planted logits to a row, none alike: up to 19 of them among the chunks of one thread, which lie
    1024 chunks apart, the others anywhere."""
    rng = np.random.default_rng(V)
    width = 4 if dtype == "f32" else 8            # elements of 16 bytes
    per = V // (width * THREADS)                  # chunks that every thread has
    planted = np.zeros((ROWS, 24), dtype=np.int64)
    for row in range(ROWS):
        together = row % 20                       # of the 24, so many in one thread
        thread, there = rng.integers(0, THREADS), rng.permutation(per * width)[:together]
        mine = (thread + there // width * THREADS) * width + there % width
        others = rng.permutation(V)[:100]
        others = others[~np.isin(others, mine)][:24 - len(mine)]
        planted[row] = rng.permutation(np.concatenate([mine, others]))
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.rand(ROWS, V, device="cuda", generator=gen)
    at = torch.from_numpy(planted).cuda()
    x.scatter_(1, at, torch.arange(25, 1, -1, device="cuda", dtype=torch.float32).expand(ROWS, 24))
    x = x.to(dtype_of(torch, dtype))
    print(f"[beam lists] {dtype} {V}", flush=True)
    for top in (1, 5, 16, 24):
        for _ in range(3):
            assert torch.equal(step(torch, x, top).tokens[:, :24], at[:, :top])


@pytest.mark.parametrize("values", [1, 2, 3, 50])
@pytest.mark.parametrize("V", [70008, 90001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_distinct_logits(torch, dtype, V, values):
    gen = torch.Generator(device="cuda").manual_seed(values)
    x = torch.randint(0, values, (ROWS, V), device="cuda", generator=gen).to(dtype_of(torch, dtype))
    x[::7, 17:] = -1                              # and rows with few of them
    order = x.float().sort(dim=1, descending=True, stable=True).indices
    print(f"[beam lists] {dtype} {V} of {values} values", flush=True)
    for top in (3, 64):
        first = step(torch, x, top)
        assert torch.equal(first.tokens, order[:, :top])
        for _ in range(2):
            assert all(torch.equal(a, b) for a, b in zip(step(torch, x, top), first))
