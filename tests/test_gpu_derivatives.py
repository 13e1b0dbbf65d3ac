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


U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def far_rows(torch, dtype, V, gen):
    """Rows whose log-sum-exp is far from 0: offsets, and masks of nothing but the type's lowest value."""
    low = torch.finfo(dtype).min
    x = torch.randn(7, V, device="cuda", generator=gen)
    x[0] = low                                     # every token masked
    x[1] = x[1].mul(2).round() + 60000
    x[2] = x[2].mul(2).round() - 30000
    x[3, 1:] = low                                 # all but one
    x[4] = 60000.0
    x[5] = x[5] + 1000
    return x.clamp(min=low).to(dtype)


@pytest.mark.parametrize("dt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V,rows", [(11, 1), (5000, 1), (70001, 1), (300, 90)])
def test_gradient_of_rows_far_from_zero(torch, dt, V, rows):
    """softmax's probabilities through autograd, whatever the logits' size: p off by
    (3 |log p| + 8) U relative, log p by as much as the logsumexp's tolerance, then the type's step."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = far_rows(torch, getattr(torch, dt), V, gen).repeat(rows, 1).requires_grad_()
    M = x.shape[0]
    tok = torch.randint(0, V, (M,), device="cuda", generator=gen)
    tok[6::7] = -1
    k, h, s = (torch.randn(M, device="cuda", generator=gen) for _ in range(3))
    print(f"[far rows] {M}x{V} {dt}", flush=True)
    r = g.token_logprobs(x, tok)
    (k * r.logprobs + h * r.entropy + s * r.lse).sum().backward()
    y = x.detach().double()
    logp = y.log_softmax(1)
    p = logp.exp()
    given = (tok >= 0).double()[:, None]
    hot = torch.nn.functional.one_hot(tok.clamp_min(0), V) * given
    # p log p is 0 where p is; log p of masked tokens is -1e38 and stays out of the sums
    lg = torch.where(p > 0, logp, 0.0)
    ent = -(p * lg).sum(1, keepdim=True)
    k, h, s = (t.double()[:, None] for t in (k, h, s))
    want = k * (hot - given * p) - h * p * (lg + ent) + s * p
    size = p * (k.abs() + s.abs()) + h.abs() * p * (lg.abs() + ent)
    sums = (64 + V / 256 + 32) * 2 * U             # of the row's log-sum, as in the forward tests
    tol = size * ((3 * lg.abs() + 8) * U + sums) + h.abs() * p * sums * (2 * torch.tensor(float(V)).log() + 2)
    tol = tol + (k * hot).abs() * U
    tol = tol + HALF[dt] * (want.abs() + tol) + {"float32": 2.0 ** -126, "bfloat16": 2.0 ** -126,
                                                 "float16": 2.0 ** -25}[dt]
    worst = ((x.grad.double() - want).abs() - tol).amax(1)
    assert (worst <= 0).all(), worst
    # and by a direct call with what the forward left off, in either layer's way in
    M, V = x.shape
    low = torch.full((M,), float("nan"), device="cuda")
    lp, lse, entropy = (torch.empty(M, device="cuda") for _ in range(3))
    code = ["float32", "bfloat16", "float16"].index(dt)
    g.token_logprobs_raw(M, V, x.data_ptr(), code, V, tok.data_ptr(), 8, lp.data_ptr(), entropy.data_ptr(),
                         lse.data_ptr(), stream=torch.cuda.current_stream().cuda_stream, lse_low=low.data_ptr())
    assert (low[lse.abs() < 64] == 0).all() and torch.isfinite(low).all()
    gk, gh, gs = (t[:, 0].float() for t in (k, h, s))
    for out in (None, torch.empty_like(x)):
        d = g.token_logprobs_backward(x.detach(), tok, lse, entropy, gk, gh, gs, out=out, lse_low=low)
        worst = ((d.double() - want).abs() - tol).amax(1)
        assert (worst <= 0).all(), worst


def test_gradient_of_empty_and_undefined_rows(torch):
    """Rows of -infinity, with a NaN, with an infinity, through autograd: as by a direct call."""
    x = torch.randn(4, 1000, device="cuda")
    x[0], x[1, 3], x[2, 5] = float("-inf"), float("nan"), float("inf")
    x.requires_grad_()
    tok = torch.tensor([1, 2, 3, 4], device="cuda")
    r = g.token_logprobs(x, tok)
    (r.logprobs + r.entropy + r.lse).sum().backward()
    assert (x.grad[0] == 0).all() and x.grad[1:3].isnan().all() and x.grad[3].isfinite().all()
