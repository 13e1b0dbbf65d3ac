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


def test_tangents_are_refused():
    """No operator of decoding has a forward-mode derivative; a tangent is not dropped unseen."""
    torch = pytest.importorskip("torch")
    fa = torch.autograd.forward_ad
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    beams, bias = torch.zeros(1, 2, dtype=torch.int64), torch.zeros(2)
    with fa.dual_level():
        def dual(t):
            return fa.make_dual(t, torch.ones_like(t))
        for call in (lambda: g.quantize_mx4(dual(x)), lambda: g.linear_mx4(dual(x), q, s),
                     lambda: g.linear_mx4(dual(x[None]), q, s), lambda: g.matmul_mx4(q, s, q, s, bias=dual(bias)),
                     lambda: g.dequantize_mx4(q, s, out=dual(x)), lambda: g.matmul_mx4(q, s, q, s, out=dual(x[:, :2])),
                     lambda: g.beam_step(dual(x), torch.zeros(1, 2)), lambda: g.beam_step(x, dual(torch.zeros(1, 2))),
                     lambda: g.reorder_beams([x, dual(x)], beams), lambda: g.reorder_beams(dual(x), beams),
                     lambda: g.reorder_beams([x], beams, out=[dual(x)])):
            with pytest.raises(NotImplementedError):
                call()
        for call in (lambda: g.quantize_mx4(x), lambda: g.linear_mx4(x, q, s), lambda: g.beam_step(x, torch.zeros(1, 2)),
                     lambda: g.reorder_beams([x], beams)):
            with pytest.raises(ValueError):                      # not on a GPU
                call()
