"""Derivatives the operators do not have are refused, not dropped (on a host without a GPU)."""
import pytest

import fp32_gemm_f32_amd as g


def test_token_logprobs_refuses_a_tangent():
    torch = pytest.importorskip("torch")
    fa = torch.autograd.forward_ad
    x, tok = torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64)
    with fa.dual_level():
        dual = fa.make_dual(x, torch.ones(2, 4))
        with pytest.raises(NotImplementedError):
            g.token_logprobs(dual, tok)
        with pytest.raises(NotImplementedError):
            g.token_logprobs(dual.t().contiguous().t(), tok, top=2)
        with pytest.raises(ValueError):
            g.token_logprobs(x, tok)                         # not on a GPU
    with pytest.raises(ValueError):
        g.token_logprobs(x, tok)


def test_refusals_of_lse_low():
    """Misaligned or overlapping, before any HIP call (addresses that nothing reads)."""
    P, STEP = 1 << 20, 1 << 16
    at = [P + i * STEP for i in range(10)]
    lib = g.library()

    def forward(low):
        return lib.token_logprobs_low(4, 100, at[0], 1, 100, at[1], 8, at[2], at[3], at[4], low, 2, at[5], at[6],
                                      None, 0, None)

    def backward(low, dx):
        return lib.token_logprobs_backward_low(4, 100, at[0], 1, 100, at[1], 8, at[2], low, at[3], at[4], at[5],
                                               at[6], dx, 100, None)
    PTR, ALIAS = -3, -4
    assert forward(at[7] + 2) == PTR
    assert forward(at[0]) == ALIAS and forward(at[4] + 12) == ALIAS and forward(at[6] + 60) == ALIAS
    assert backward(at[7] + 1, at[8]) == PTR
    assert backward(at[8], at[8]) == ALIAS and backward(at[8] + 796, at[8]) == ALIAS
