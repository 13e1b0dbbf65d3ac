"""Keys and values that are slices of one cache, reordered in place together."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g
from test_gpu_beams import chosen, moved

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


# the cache's shape behind its rows (or, rows=1, behind a dimension before them), and which dimension holds the
# two
LAYOUTS = [((2, 9, 3, 8), 1, 0), ((9, 2, 3, 8), 2, 0), ((9, 3, 2, 8), 3, 0), ((9, 3, 8, 2), 4, 0), ((9, 2, 3, 7), 2, 0),
           ((2, 3, 8), 2, 1), ((3, 2, 5), 3, 1)]


@pytest.mark.parametrize("B,W", [(1, 1), (1, 4), (3, 5), (2, 64)])
@pytest.mark.parametrize("shape,at,rows_at", LAYOUTS)
def test_two_slices_of_a_cache(torch, B, W, shape, at, rows_at):
    rng = np.random.default_rng(W)
    beams = chosen(rng, B, W)
    n = B * W
    full = (n, *shape) if rows_at == 0 else (6, n, *shape)
    cache = torch.randn(full, device="cuda", dtype=torch.bfloat16)
    parts = [cache.select(at, i).movedim(rows_at, 0) for i in range(2)]
    want = [moved(torch, t, beams) for t in parts]
    dev = torch.from_numpy(beams).cuda()
    print(f"[slices] {B}x{W} {full} {at}", flush=True)
    back = g.reorder_beams(parts, dev, out=parts)
    assert all(a is b for a, b in zip(back, parts))
    for a, b in zip(parts, want):
        assert torch.equal(a.cpu(), b)


def test_live_positions_alone(torch):
    """The first positions of a cache that holds more: the others stay as they are."""
    cache = torch.randn(8, 20, 2, 4, 16, device="cuda")
    before, beams = cache.clone(), np.array([[1, 1, 0, 2], [3, 0, -1, 3]])
    live = [cache[:, :11, i] for i in range(2)]
    g.reorder_beams(live, torch.from_numpy(beams).cuda(), out=live)
    assert torch.equal(cache[:, 11:], before[:, 11:])
    assert torch.equal(cache[:, :11].cpu(), moved(torch, before, beams)[:, :11])
    # a part of one that reaches into the other is refused
    flat = cache.view(8, 20, -1)
    with pytest.raises(g.SgemmError) as e:
        g.reorder_beams([flat[:, :, :65], flat[:, :, 64:]], torch.from_numpy(beams).cuda(),
                        out=[flat[:, :, :65], flat[:, :, 64:]])
    assert e.value.status == -4
