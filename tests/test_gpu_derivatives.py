"""Derivatives of the token log-probabilities: forward mode is refused, not dropped."""
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


@pytest.mark.parametrize("grad", [False, True])
def test_a_tangent_is_refused(torch, grad):
    fa = torch.autograd.forward_ad
    x = torch.randn(3, 50, device="cuda", requires_grad=grad)
    tok = torch.tensor([1, -1, 49], device="cuda")
    want = g.token_logprobs(x, tok)
    with fa.dual_level():
        dual = fa.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError):                    # NotImplementedError is one
            g.token_logprobs(dual, tok, top=2)
        assert torch.equal(g.token_logprobs(x, tok).logprobs, want.logprobs)
        assert torch.equal(g.token_logprobs(fa.unpack_dual(dual).primal.detach(), tok).lse, want.lse)
    assert torch.equal(g.token_logprobs(x, tok).lse, want.lse)
