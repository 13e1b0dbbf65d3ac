"""Forms of the 8-bit product that its plan takes for large or ragged operands: copies into place, splits
of copies, results stored past the caches, and the same bits from every one of them."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def codes(torch, rows, cols, ld, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, (rows, ld), dtype=torch.int8, device="cuda", generator=gen)[:, :cols]


def exact_sums(torch, a, b):
    """The integer sums, as 64-bit floats (far below 2^53)."""
    return torch.matmul(a.double(), b.double().t().contiguous())


def definition(sums, sa, sb, bias, dtype):
    """The header's roundings: the sum to FP32, the scales' product, one of both the scaling and the
    bias (in 64 bits the product of two FP32 numbers is exact, and adding the bias there first moves
    what the second rounding sees by 2^-53 relative), and C's type."""
    s, scale = sums.float(), sa[:, None] * sb
    return (s.double() * scale.double() + bias.double()).float().to(dtype)


@pytest.mark.parametrize("M,N,K", [(96, 80, 16384), (9, 70, 65536), (700, 690, 8000), (300, 5000, 4095), (3, 500, 777)])
@pytest.mark.parametrize("dt", DTYPES)
def test_every_form_rounds_alike(torch, M, N, K, dt):
    """With a bias: split and whole, from the tiles and the join, to the bit."""
    a, b = codes(torch, M, K, K, 1), codes(torch, N, K, K, 2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    sa, sb = (torch.rand(n, device="cuda", generator=gen) * 0.01 + 1e-4 for n in (M, N))
    bias = torch.randn(N, device="cuda", generator=gen) * 3
    dtype = dtype_of(torch, dt)
    print(f"[i8 forms] {M}x{N}x{K} {dt}", flush=True)
    c = g.matmul_i8(a, sa, b, sb, bias=bias, out_dtype=dtype)
    d = torch.empty_like(c)
    g.gemm_i8(M, N, K, a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), K, sb.data_ptr(), bias.data_ptr(),
              d.data_ptr(), DTYPES.index(dt), N, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(c, d)
    want = definition(exact_sums(torch, a, b), sa, sb, bias, dtype)
    # the oracle's two roundings (53 bits, then 24) may differ from one where they meet a tie: one
    # element in 2^29 or so, and by one step
    off = c != want
    assert off.sum() <= 1, f"{int(off.sum())} of {off.numel()} elements differ"
