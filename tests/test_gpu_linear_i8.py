"""The 8-bit projection on activations of any number of dimensions, empty ones too."""
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(7,), (3, 7), (2, 3, 7), (0, 7), (2, 0, 7), (0,), (3, 0), (2, 3, 0), (0, 3, 0)])
@pytest.mark.parametrize("bias", [False, True])
def test_shapes(shape, bias):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N, K = 5, shape[-1]
    w, scales = g.quantize_rows(torch.randn(N, K, device="cuda"))
    x = torch.randn(shape, device="cuda")
    b = torch.randn(N, device="cuda") if bias else None
    print(f"[linear] {shape}", flush=True)
    y = g.linear_i8(x, w, scales, bias=b, out_dtype=torch.float32)
    assert y.shape == (*shape[:-1], N)
    rows = 1
    for n in shape[:-1]:
        rows *= n
    flat = x.reshape(rows, K)
    q, s = g.quantize_rows(flat)
    want = q.double() @ w.double().t().contiguous() * s.double()[:, None] * scales.double()
    want = want + (b.double() if bias else 0.0)
    size = want.abs() + (b.abs() if bias else 0.0)
    assert ((y.reshape(rows, N).double() - want).abs() <= 8 * 2.0 ** -24 * size + 1e-30).all()
