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
