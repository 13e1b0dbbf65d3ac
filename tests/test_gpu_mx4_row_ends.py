"""Rows whose last block of 32 ends in the middle: the 4-bit quantiser writes a row's bytes and no other,
with rows packed one behind another and with bytes between them, through every way in."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g
import mx4_util as mx
from test_gpu_gemm_i8 import assert_guard, dtype_of, guarded

pytestmark = pytest.mark.gpu

TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


# a row of K elements has units of 8 up to the block's end: with 7, 15 and 23 over whole blocks one of
# them starts one element behind the row; packed rows of 4 n bytes follow each other. The last two
# are quantised several units to a thread.
SHAPES = [(1, 7), (128, 7), (300, 15), (65, 23), (64, 39), (300, 47), (33, 55), (5, 4087), (3, 4103), (70, 9),
          (70, 17), (70, 25), (70, 30), (70, 41), (2049, 4103), (131080, 39)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_end_where_they_end(torch, dtype, M, K):
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K))
    x[:, :2] += np.sign(x[:, :2]) * 2                     # the first two codes of a row are not 0
    t = torch.from_numpy(x).to(dtype_of(torch, dtype))
    row, nb = (K + 1) // 2, (K + 31) // 32
    codes, scales = mx.quantize(t.double().numpy())
    want = torch.from_numpy(mx.pack(codes)), torch.from_numpy(scales)
    dx = t.cuda()
    print(f"[mx4 row ends] {dtype} {M}x{K}", flush=True)
    for pad in (0, 1, 5):
        raw_q, q = guarded(torch, M, row, row + pad, torch.uint8)
        raw_s, s = guarded(torch, M, nb, nb + pad, torch.uint8)
        g.quantize_mx4(dx, out=q, scales=s)
        assert torch.equal(q.cpu(), want[0]) and torch.equal(s.cpu(), want[1]), pad
        assert_guard(raw_q, q, M, row, row + pad)
        assert_guard(raw_s, s, M, nb, nb + pad)
    for _ in range(3):
        q, s = g.quantize_mx4(dx)
        assert torch.equal(q.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
    values = torch.from_numpy(mx.values(codes, scales)).to(t.dtype)
    assert torch.equal(g.dequantize_mx4(q, s, dtype=t.dtype, columns=K).cpu(), values)


@pytest.mark.parametrize("M,N,K", [(1, 64, 7), (20, 70, 39), (300, 130, 55), (33, 257, 1047)])
def test_projection_of_odd_rows(torch, M, N, K):
    """Activations and weights of an odd K: the values are those of the definition, whose products with
    scales of a few steps FP32 sums exactly."""
    rng = np.random.default_rng(K)
    x, w = (rng.integers(-6, 7, size=(r, K)).astype(np.float32) for r in (M, N))
    y = g.linear_mx4(torch.from_numpy(x).cuda(), *g.quantize_mx4(torch.from_numpy(w).cuda()))
    a, b = mx.values(*mx.quantize(x)), mx.values(*mx.quantize(w))
    want = a @ b.T
    # products are multiples of 2^-4 (codes of 0.5, scales of 2^-1 at least) and at most 36: sums take 23 bits
    assert (np.abs(a) @ np.abs(b).T).max() * 16 * 4 < 2 ** 24
    np.testing.assert_array_equal(y.cpu().numpy(), want.astype(np.float32))
