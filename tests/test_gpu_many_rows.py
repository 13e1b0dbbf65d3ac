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


def test_logprobs(torch):
    M, V, top = ITEMS // 256 + 1029, 5, 2          # a row to a workgroup of 256
    x = torch.empty(M, V, dtype=torch.float16, device="cuda").normal_()
    tok = torch.arange(M, dtype=torch.int32, device="cuda") % 7 - 1        # some below 0, some past V
    print(f"[many rows] logprobs {M}x{V}", flush=True)
    r = g.token_logprobs(x, tok, top=top)
    for w in windows(ITEMS // 256, M):
        one = g.token_logprobs(x[w].contiguous(), tok[w].contiguous(), top=top)
        for name, a, b in zip(one._fields, r, one):
            assert torch.equal(a[w].nan_to_num(7.0), b.nan_to_num(7.0)), name
        want = x[w].double().log_softmax(1)
        given = (tok[w] >= 0) & (tok[w] < V)
        at = want[given].gather(1, tok[w][given].long()[:, None])[:, 0]
        # (logs of sums of five terms: a few steps of FP32)
        assert (r.logprobs[w][given].double() - at).abs().max() <= 32 * 2.0 ** -24 * 8
        assert torch.equal(r.logprobs[w].isnan(), tok[w] >= V) and (r.logprobs[w][tok[w] < 0] == 0).all()


def test_gradient(torch):
    M, V = ITEMS // 256 + 1029, 5                  # a row to a workgroup of 256
    x = torch.empty(M, V, dtype=torch.float16, device="cuda").normal_()
    out = torch.full((M, V), 99.0, dtype=torch.float16, device="cuda")
    tok = torch.arange(M, device="cuda") % 6 - 1
    r = g.token_logprobs(x, tok)
    k = torch.rand(M, device="cuda")
    print(f"[many rows] gradient {M}x{V}", flush=True)
    g.token_logprobs_backward(x, tok, r.lse, r.entropy, k, k, out=out)
    for w in windows(ITEMS // 256, M):
        rows = [t[w].contiguous() for t in (x, tok, r.lse, r.entropy, k, k)]
        assert torch.equal(out[w], g.token_logprobs_backward(*rows))
        given = (tok[w] >= 0)[:, None]
        hot = torch.nn.functional.one_hot(tok[w].clamp_min(0), V) * given
        logp = x[w].double().log_softmax(1)
        p = logp.exp()
        h = -(p * logp).sum(1, keepdim=True)
        want = k[w].double()[:, None] * (hot - p * given - p * (logp + h))
        # values of up to 3 or so: half a step of FP16, and sums of a few terms in FP32
        assert (out[w].double() - want).abs().max() <= 4 * 2.0 ** -11


def product_reference(a, sa, b, sb, bias):
    """The definition for few columns of K: exact sums, and the size its roundings are relative to."""
    s = (a.double()[:, None, :] * b.double()[None, :, :]).sum(2)
    scaled = s * sa.double()[:, None] * sb.double()
    return scaled + bias.double(), scaled.abs() + bias.double().abs()


def test_few_rows_by_many_columns(torch):
    M, K = 2, 16
    border = ITEMS // 512 * 16                     # 16 columns to a workgroup of 512
    N = border + 1029
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    b = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    sa, sb, bias = torch.rand(M, device="cuda"), torch.rand(N, device="cuda"), torch.randn(N, device="cuda") * 1e4
    out = torch.full((M, N), float("nan"), device="cuda")
    print(f"[many columns] product {M}x{N}x{K}", flush=True)
    g.matmul_i8(a, sa, b, sb, bias=bias, out=out)
    for w in windows(border, N):
        want, size = product_reference(a, sa, b[w], sb[w], bias[w])
        assert ((out[:, w].double() - want).abs() <= 5 * 2.0 ** -24 * size).all()
    assert torch.isfinite(out).all()


def test_tiles_of_many_columns(torch):
    M, K = 17, 1
    border = 1 << 30                               # what one launch takes of them
    N = border + 1029
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    b = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    print(f"[many columns] product {M}x{N}x{K}", flush=True)
    g.gemm_i8(M, N, K, a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), K, sb.data_ptr(), 0, out.data_ptr(), 1, N,
              stream=torch.cuda.current_stream().cuda_stream)
    for w in windows(border, N):
        s = a.float() * b[w].float().t()
        assert torch.equal(out[:, w], (s * (sa[:, None] * sb[w])).to(torch.bfloat16))


def test_tiles_of_many_rows(torch):
    """As many rows as an int counts: the last tile reaches past them."""
    M, N, K = 2 ** 31 - 5, 2, 1
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    b = torch.tensor([[3], [-5]], dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    print(f"[many rows] product {M}x{N}x{K}", flush=True)
    g.gemm_i8(M, N, K, a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), K, sb.data_ptr(), 0, out.data_ptr(), 1, N,
              stream=torch.cuda.current_stream().cuda_stream)
    for w in windows(1 << 30, M):
        s = a[w].float() * b.float().t()
        assert torch.equal(out[w], (s * (sa[w, None] * sb)).to(torch.bfloat16))
