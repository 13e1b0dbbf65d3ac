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


def run_and_check(torch, M, N, K, lda, ldb, dt, seed):
    """Against exact sums, into rows of exactly N elements, with a bias; then without a workspace,
    to the same bits."""
    a, b = codes(torch, M, K, lda, seed), codes(torch, N, K, ldb, seed + 1)
    gen = torch.Generator(device="cuda").manual_seed(seed + 2)
    sa, sb = (torch.rand(n, device="cuda", generator=gen) * 0.01 + 1e-4 for n in (M, N))
    bias = torch.randn(N, device="cuda", generator=gen)
    dtype = dtype_of(torch, dt)
    c = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    g.matmul_i8(a, sa, b, sb, bias=bias, out=c)
    want = definition(exact_sums(torch, a, b), sa, sb, bias, dtype)
    off = c != want
    # (as in test_every_form_rounds_alike: the oracle rounds twice, one element in 2^29 or so)
    assert off.sum() <= 1, f"{int(off.sum())} of {off.numel()} elements differ"
    d = torch.full_like(c, float("nan"))
    g.gemm_i8(M, N, K, a.data_ptr(), lda, sa.data_ptr(), b.data_ptr(), ldb, sb.data_ptr(), bias.data_ptr(),
              d.data_ptr(), DTYPES.index(dt), N, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(c, d)
    # and through the extension, whose output is its own
    assert torch.equal(g.matmul_i8(a, sa, b, sb, bias=bias, out_dtype=dtype), c)


COPIES = [(1078, 14336, 64, 5, 0, [True, False], False), (1920, 8320, 128, 0, 3, [False, True], False),
          (3287, 11456, 101, 0, 0, [True, True], False), (2496, 192, 12416, 0, 3, [False, True], True),
          (258, 1550, 12720, 13, 0, [True, False], True), (2875, 135, 12560, 0, 13, [False, True], True)]


@pytest.mark.parametrize("M,N,K,pad_a,pad_b,copies,split", COPIES)
@pytest.mark.parametrize("dt", DTYPES)
def test_copies_into_place(torch, M, N, K, pad_a, pad_b, copies, split, dt):
    """Operands off the alignment the tiles load are copied to the workspace: A, B, both, and with K
    split behind it."""
    d = g.gemm_i8_plan_describe(M, N, K, K + pad_a, K + pad_b, num_cus=256)
    assert d["copies"] == copies and (d["splits"] > 1) == split
    print(f"[i8 copies] {M}x{N}x{K} ld +{pad_a} +{pad_b} {dt}", flush=True)
    run_and_check(torch, M, N, K, K + pad_a, K + pad_b, dt, M)


# one for each tile and form, with one round of workgroups and with several (of the forms that go on to
# another tile: those do); every row of C starts on a line of 64 bytes, so results go past the caches
TIGHT = [(143, 5824, 144), (4762, 832, 128), (263, 6976, 656), (6740, 1024, 2976), (325, 6016, 129),
         (6791, 1152, 1219), (3309, 1216, 288), (3084, 5056, 928), (6967, 576, 147), (3247, 5056, 131),
         (1057, 7232, 656), (3480, 5952, 400), (906, 7424, 417), (2393, 7616, 403), (1681, 4864, 128),
         (3610, 5760, 128), (3500, 5824, 272), (6179, 960, 131), (2532, 7552, 131), (349, 2752, 929),
         (536, 6976, 1025), (341, 2880, 288), (642, 5696, 144), (132, 6272, 131), (562, 6912, 129),
         (8763, 64, 704), (77, 192, 135), (39, 256, 176), (5560, 320, 304), (66, 5248, 163), (4121, 448, 177),
         (19, 4992, 2771), (25, 64, 1936), (16, 4096, 512), (9, 64, 300)]


@pytest.mark.parametrize("M,N,K", TIGHT)
@pytest.mark.parametrize("dt", DTYPES)
def test_rows_of_whole_lines(torch, M, N, K, dt):
    print(f"[i8 lines] {M}x{N}x{K} {dt}", flush=True)
    run_and_check(torch, M, N, K, K, K, dt, M + N)
