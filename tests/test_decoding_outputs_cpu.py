"""Outputs that a caller gives to the decoding operators, and autograd (on a host without a GPU)."""
import pytest

import fp32_gemm_f32_amd as g


def test_outputs_that_require_grad_are_refused():
    torch = pytest.importorskip("torch")
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    beams = torch.zeros(1, 2, dtype=torch.int64)
    leaf = torch.zeros(2, 64, requires_grad=True)
    for out in (leaf, leaf * 2, torch.nn.Parameter(x)):
        for call in (lambda: g.matmul_mx4(q, s, q, s, out=out), lambda: g.dequantize_mx4(q, s, out=out),
                     lambda: g.reorder_beams([x], beams, out=[out]), lambda: g.reorder_beams(x, beams, out=out)):
            with pytest.raises(RuntimeError, match="requires grad"):
                call()
            with torch.no_grad(), pytest.raises(ValueError):     # not on a GPU
                call()
