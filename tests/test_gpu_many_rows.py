"""Operators over more rows or columns than one launch may have workgroups for (HIP takes fewer than
2^32 work items in a dimension): every row and column is served, on both sides of a launch's border."""
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu

ITEMS = 2 ** 32 - 1


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    yield t
    t.cuda.empty_cache()


def windows(border, n, rows=1 << 16):
    """Where to look: the start, both sides of the border, the end."""
    assert border < n, "the case is meant to need a second launch"
    return [slice(0, rows), slice(border - rows, min(n, border + rows)), slice(n - 40, n)]


def test_quantize(torch):
    K = 3
    border = ITEMS // 256 * 32                     # 32 such rows to a workgroup of 256
    M = border + 1029
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((M,), -1.0, device="cuda")
    print(f"[many rows] quantize {M}x{K}", flush=True)
    g.quantize_rows(x, out=q, scales=scales)
    assert (scales >= 0).all()
    for w in windows(border, M):
        # each division rounded once: in 64 bits, then to 32
        peak = x[w].float().abs().amax(1).double()
        assert torch.equal(scales[w], (peak / 127).float())
        inverse = (127 / peak).float()
        assert torch.equal(q[w], (x[w].float() * inverse[:, None]).round().clamp(-127, 127).to(torch.int8))
