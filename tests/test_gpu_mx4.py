"""Microscaled 4-bit floating point against numpy in 64 bits, through the C ABI and the tensor layer:
the quantiser and its inverse to the bit, the product exactly where its sums fit FP32 and within
counted roundings elsewhere; odd sizes, strides and addresses, edge blocks, other streams and graph
capture."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g
import mx4_util as mx
from test_gpu_gemm_i8 import assert_guard, dtype_of, guarded, strided

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # half a step, relative
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def operand(rng, rows, cols, low=126, high=128):
    """Random codes and scales within [low, high]."""
    return (rng.integers(0, 16, size=(rows, cols)).astype(np.uint8),
            rng.integers(low, high + 1, size=(rows, -(-cols // 32))).astype(np.uint8))


def on_gpu(torch, host, ld=None, offset=0, fill=0xff):
    """Bytes in a GPU buffer of rows of ld after `offset`; the others are `fill` (as scales: NaN)."""
    return strided(torch, torch.from_numpy(host), host.shape[1] if ld is None else ld, offset, fill)[1]


# ------------------------------------------------------------------ the quantiser -------

@pytest.mark.parametrize("M,K,pad,offset", [(1, 1, 0, 0), (3, 31, 0, 1), (5, 32, 3, 0), (2, 33, 0, 1),
                                            (7, 63, 1, 3), (16, 256, 0, 0), (33, 1000, 5, 1), (4, 4099, 0, 0),
                                            (300, 72, 8, 0), (2, 70000, 0, 0), (2049, 5, 0, 1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(torch, dtype, M, K, pad, offset):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((M, K)) * np.exp(2 * rng.standard_normal((M, 1)))
    x[:, ::3] = np.round(x[:, ::3] * 4) / 4               # many on the borders between codes
    t = torch.from_numpy(x).to(dtype_of(torch, dtype))
    _, dx = strided(torch, t, K + pad, offset, 1e30 if dtype != "f16" else 6e4)
    row, nb = (K + 1) // 2, (K + 31) // 32
    raw_q, q = guarded(torch, M, row, row + pad, torch.uint8)
    raw_s, s = guarded(torch, M, nb, nb + pad, torch.uint8)
    print(f"[mx4 quantize] {dtype} {M}x{K}", flush=True)
    g.quantize_mx4(dx, out=q, scales=s)
    codes, scales = mx.quantize(t.double().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.cpu().numpy(), mx.pack(codes))
    assert_guard(raw_q, q, M, row, row + pad)
    assert_guard(raw_s, s, M, nb, nb + pad)
    q2, s2 = g.quantize_mx4(dx)
    assert torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_16_bit_number(torch, dtype):
    """Each number as a block's largest, beside its halves, quarters, ..., and the borders between
    codes over it."""
    bits = np.arange(65536, dtype=np.uint16)
    if dtype == "f16":
        base = bits.view(np.float16).astype(np.float64)
    else:
        with np.errstate(invalid="ignore"):
            base = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    parts = np.array([1, 0.5, 0.25, 0.125, 0.0625, 0.75, 0.375, 0.1875, -1, -0.5, -0.625, 1 / 3, -1 / 7, 1e-3, 0, -0.0])
    with np.errstate(invalid="ignore"):
        x = np.concatenate([base[:, None] * parts[None, :], np.zeros((65536, 16))], axis=1)
    t = torch.from_numpy(x).to(dtype_of(torch, dtype))
    codes, scales = mx.quantize(t.double().numpy())
    q, s = g.quantize_mx4(t.cuda())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.cpu().numpy(), mx.pack(codes))


def test_quantize_edge_blocks(torch):
    x = np.zeros((10, 96), dtype=np.float32)
    x[0, 40] = -0.0
    x[1, 5], x[1, 40] = np.nan, 3.0
    x[2, 64], x[2, 0] = np.inf, 1.0
    x[3, 33], x[3, 34] = -np.inf, np.nan
    x[4, 0], x[4, 1] = 3.4028235e38, -1.7e38
    x[5, 0] = 1e-45                                       # FP32's least
    x[6, 0], x[6, 1] = 2.0 ** -126, 2.0 ** -129
    x[7, 0], x[7, 1] = 2.0 ** -125, 2.0 ** -127
    x[8, :] = 1e-40
    x[9, 0] = 7.999999
    q, s = g.quantize_mx4(torch.from_numpy(x).cuda())
    codes, scales = mx.quantize(x)
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.cpu().numpy(), mx.pack(codes))
    assert scales[1].tolist() == [255, 126, 0]
    assert scales[0].tolist() == [0, 0, 0] and codes[0, 40] == 8 and codes[9, 0] == 7


# ------------------------------------------------------------------ its inverse ---------

@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(torch, dtype):
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    y = g.dequantize_mx4(on_gpu(torch, mx.pack(codes)), on_gpu(torch, scales), dtype=dtype_of(torch, dtype))
    want = torch.from_numpy(mx.values(codes, scales)).to(dtype_of(torch, dtype))
    got = y.cpu()
    assert torch.equal(got.isnan(), want.isnan()) and want[255].isnan().all()
    assert torch.equal(got[:255], want[:255])
    assert torch.equal(torch.signbit(got[:255]), torch.signbit(want[:255]))


@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (3, 31, 2), (5, 33, 0), (40, 1000, 1), (9, 2047, 0), (300, 64, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_forms(torch, dtype, M, K, pad):
    rng = np.random.default_rng(K)
    codes, scales = operand(rng, M, K, 120, 134)
    q, s = mx.pack(codes), scales
    dq, ds = on_gpu(torch, q, q.shape[1] + pad, pad), on_gpu(torch, s, s.shape[1] + pad, pad)
    want = torch.from_numpy(mx.values(codes, scales)).to(dtype_of(torch, dtype))
    raw, y = guarded(torch, M, K, K + pad, dtype_of(torch, dtype))
    g.dequantize_mx4(dq, ds, columns=K, out=y)
    assert torch.equal(y.cpu(), want)
    assert_guard(raw, y, M, K, K + pad)
    assert torch.equal(g.dequantize_mx4(dq, ds, dtype=dtype_of(torch, dtype), columns=K).cpu(), want)


# ------------------------------------------------------------------ the product ---------

# few rows, every tile and split, ragged in each dimension, K of one pair to many panels
SHAPES = [(1, 1, 2), (1, 16, 32), (3, 17, 34), (16, 16, 512), (15, 33, 1024), (1, 512, 2048), (2, 300, 8192),
          (17, 31, 66), (32, 500, 2048), (48, 1000, 1536), (64, 64, 1024), (65, 129, 1030), (128, 96, 4096),
          (127, 255, 254), (256, 256, 256), (255, 511, 510), (300, 700, 1100), (513, 1025, 2050), (1024, 512, 512),
          (33, 64, 16384), (1000, 1500, 96), (2048, 2048, 256), (700, 4100, 320)]


def exact_case(rng, M, N, K):
    """Operands whose sums FP32 holds exactly in any order: products are multiples of 2^-4 (0.25 with
    scales down to 2^-1 on both sides) and at most 36 * 4, so sums stay below 2^24 multiples up to K =
    7281; longer ones take scales of 1."""
    low, high = (126, 128) if K <= 4096 else (127, 127)
    return operand(rng, M, K, low, high), operand(rng, N, K, low, high)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("layout", ["packed", "padded", "odd"])
def test_product_is_exact(torch, M, N, K, layout):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    (ca, sa), (cb, sb) = exact_case(rng, M, N, K)
    pad, offset = {"packed": (0, 0), "padded": (16, 16), "odd": (3, 1)}[layout]
    nb = sa.shape[1]
    dA, dB = (on_gpu(torch, mx.pack(c), K // 2 + pad, offset) for c in (ca, cb))
    dsa, dsb = (on_gpu(torch, s, nb + pad, offset) for s in (sa, sb))
    raw, C = guarded(torch, M, N, N + 3, torch.float32)
    print(f"[mx4 product] {M}x{N}x{K} {layout}", flush=True)
    g.matmul_mx4(dA, dsa, dB, dsb, out=C)
    want = mx.values(ca, sa) @ mx.values(cb, sb).T
    got = C.cpu().numpy()
    assert np.abs(want).max() * 16 < 2 ** 24
    np.testing.assert_array_equal(got, want.astype(np.float32))
    assert_guard(raw, C, M, N, N + 3)


@pytest.mark.parametrize("M,N,K", [(1, 700, 4096), (5, 64, 258), (40, 333, 2048), (200, 300, 1056), (512, 1024, 8192)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_product_of_quantised_numbers(torch, dtype, with_bias, M, N, K):
    """A block's products enter the sum with one rounding each, of a unit at most (2^-23 of what is
    summed in magnitude), K / 32 of them and up to 48 where waves, splits and the bias are joined; the
    result is rounded once more."""
    rng = np.random.default_rng(K + N)
    A, B = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))), rng.standard_normal((N, K))
    (ca, sa), (cb, sb) = mx.quantize(A), mx.quantize(B)
    bias = rng.standard_normal(N).astype(np.float32) if with_bias else None
    C = g.matmul_mx4(on_gpu(torch, mx.pack(ca)), on_gpu(torch, sa), on_gpu(torch, mx.pack(cb)), on_gpu(torch, sb),
                     bias=None if bias is None else torch.from_numpy(bias).cuda(), out_dtype=dtype_of(torch, dtype))
    assert C.dtype == dtype_of(torch, dtype)
    a, b = mx.values(ca, sa), mx.values(cb, sb)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        want, size = want + bias, size + np.abs(bias)
    bound = (K / 32 + 48) * 2.0 ** -23 * size * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want)
    if dtype == "f16":
        bound = bound + 2.0 ** -25                         # below its least normal number steps do not shrink
    assert (np.abs(C.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("M,N,K", [(4, 100, 1024), (40, 64, 544), (300, 520, 1056)])
def test_nan_scales_and_extreme_ones(torch, M, N, K):
    """A block whose scale is no number makes its row (or column) NaN, others not, even where its
    codes are zeros; scales far apart cancel in the product."""
    rng = np.random.default_rng(5)
    (ca, sa), (cb, sb) = operand(rng, M, K, 120, 120), operand(rng, N, K, 134, 134)
    sa[1, -1] = 255
    ca[1, :] = 0
    sb[3, 0] = 255
    sa[2, :], sa[3, :] = 1, 200
    C = g.matmul_mx4(on_gpu(torch, mx.pack(ca)), on_gpu(torch, sa), on_gpu(torch, mx.pack(cb)), on_gpu(torch, sb))
    with np.errstate(invalid="ignore"):
        want = mx.values(ca, sa) @ mx.values(cb, sb).T
    got = C.cpu().numpy().astype(np.float64)
    nan = np.zeros((M, N), dtype=bool)
    nan[1, :] = nan[:, 3] = True
    assert np.array_equal(np.isnan(got), nan)
    np.testing.assert_array_equal(got[~nan], want.astype(np.float32)[~nan])      # each row's scales are one: exact


def test_scales_behind_a_row_do_not_count(torch):
    """A K that ends inside a panel: the bytes behind a row's scales hold NaN, those behind its
    elements anything."""
    rng = np.random.default_rng(6)
    for M, N, K in [(5, 40, 34), (70, 90, 34), (300, 300, 290), (300, 300, 802)]:
        (ca, sa), (cb, sb) = operand(rng, M, K, 127, 127), operand(rng, N, K, 127, 127)
        nb = sa.shape[1]
        C = g.matmul_mx4(on_gpu(torch, mx.pack(ca), K // 2 + 15, 0), on_gpu(torch, sa, nb + 16, 0),
                         on_gpu(torch, mx.pack(cb), K // 2 + 15, 0), on_gpu(torch, sb, nb + 16, 0))
        np.testing.assert_array_equal(C.cpu().numpy(), (mx.values(ca, sa) @ mx.values(cb, sb).T).astype(np.float32))


def test_empty(torch):
    def empty(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device="cuda")
    assert g.matmul_mx4(empty(0, 16), empty(0, 1), empty(5, 16), empty(5, 1)).shape == (0, 5)
    assert g.matmul_mx4(empty(5, 16), empty(5, 1), empty(0, 16), empty(0, 1)).shape == (5, 0)
    bias = torch.randn(7, device="cuda")
    C = g.matmul_mx4(empty(3, 0), empty(3, 0), empty(7, 0), empty(7, 0), bias=bias, out_dtype=torch.bfloat16)
    assert torch.equal(C, bias.bfloat16().expand(3, 7))
    q, s = g.quantize_mx4(torch.empty(4, 0, device="cuda"))
    assert q.shape == (4, 0) and s.shape == (4, 0) and g.dequantize_mx4(q, s).shape == (4, 0)
    q, s = g.quantize_mx4(torch.empty(0, 9, device="cuda"))
    assert q.shape == (0, 5) and s.shape == (0, 1)
    w, ws = g.quantize_mx4(torch.randn(6, 64, device="cuda"))
    assert g.linear_mx4(torch.empty(2, 0, 64, device="cuda"), w, ws).shape == (2, 0, 6)


@pytest.mark.parametrize("M,N,K", [(1, 50, 64), (19, 77, 500), (33, 64, 501), (200, 1000, 1056)])
@pytest.mark.parametrize("dtype", TYPES)
def test_linear(torch, dtype, M, N, K):
    """Both steps in one call give what they give one after the other, and what their definition
    says."""
    rng = np.random.default_rng(N)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dtype_of(torch, dtype)).cuda()
    w, ws = g.quantize_mx4(torch.from_numpy(rng.standard_normal((N, K))).float().cuda())
    bias = torch.randn(N, device="cuda")
    y = g.linear_mx4(x, w, ws, bias=bias)
    q, s = g.quantize_mx4(x)
    assert y.dtype == x.dtype and torch.equal(y, g.matmul_mx4(q, s, w, ws, bias=bias, out_dtype=x.dtype))
    assert torch.equal(g.linear_mx4(x[None], w, ws, bias=bias, out_dtype=torch.float32)[0],
                       g.matmul_mx4(q, s, w, ws, bias=bias))
    a = mx.values(*mx.quantize(x.double().cpu().numpy()))
    b = mx.values(mx.unpack(w.cpu().numpy(), K), ws.cpu().numpy())
    h = bias.double().cpu().numpy()
    bound = (K / 32 + 48) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T + np.abs(h))
    want = a @ b.T + h
    assert (np.abs(g.matmul_mx4(q, s, w, ws, bias=bias).double().cpu().numpy() - want) <= bound + 2.0 ** -24 * np.abs(want)).all()


def test_other_layouts_and_refusals(torch):
    rng = np.random.default_rng(4)
    (ca, sa), (cb, sb) = operand(rng, 24, 96, 127, 127), operand(rng, 40, 96, 127, 127)
    A, B = torch.from_numpy(mx.pack(ca)).cuda(), torch.from_numpy(mx.pack(cb)).cuda()
    SA, SB = torch.from_numpy(sa).cuda(), torch.from_numpy(sb).cuda()
    want = torch.from_numpy((mx.values(ca, sa) @ mx.values(cb, sb).T).astype(np.float32))
    assert torch.equal(g.matmul_mx4(A.t().contiguous().t(), SA[:1].expand(24, 3), B, SB).cpu(), want)
    bias = torch.randn(1, device="cuda").expand(40)
    assert torch.equal(g.matmul_mx4(A, SA, B, SB, bias=bias).cpu(), want + bias.cpu())
    with pytest.raises(ValueError):
        g.matmul_mx4(A, SA[:, :2], B, SB)
    with pytest.raises(ValueError):
        g.matmul_mx4(A, SA[:23], B, SB)
    with pytest.raises(ValueError):
        g.matmul_mx4(A[:, 16:], SA[:, 1:], B, SB)
    with pytest.raises(TypeError):
        g.matmul_mx4(A.view(torch.int8), SA, B, SB)
    with pytest.raises(TypeError):
        g.matmul_mx4(A, SA, B, SB, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        g.matmul_mx4(A, SA, B, SB, out=torch.empty(24, 41, device="cuda"))
    with pytest.raises(ValueError):
        g.matmul_mx4(A, SA, B, SB, bias=torch.zeros(39, device="cuda"))
    with pytest.raises(ValueError):
        g.matmul_mx4(A, SA, B.cpu(), SB.cpu())
    with pytest.raises(ValueError):
        g.dequantize_mx4(A, SA, columns=94)
    with pytest.raises(ValueError):
        g.dequantize_mx4(A, SA, columns=-1)
    with pytest.raises(ValueError):
        g.linear_mx4(torch.zeros(2, 94, device="cuda"), B, SB)
    with pytest.raises(TypeError):
        g.quantize_mx4(torch.zeros(2, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        g.quantize_mx4(torch.zeros(2, 64, device="cuda"), out=torch.empty(2, 33, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (96, 80, 16384), (300, 280, 528), (65, 66, 68), (1024, 1024, 512)])
def test_graph_capture_and_other_stream(torch, M, N, K):
    x = torch.randn(M, K, device="cuda")
    w, ws = g.quantize_mx4(torch.randn(N, K, device="cuda"))
    want = g.linear_mx4(x, w, ws)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    print(f"[mx4 graph] {M}x{N}x{K}", flush=True)
    with torch.cuda.stream(stream):
        assert torch.equal(g.linear_mx4(x, w, ws), want)
        with torch.cuda.graph(graph, stream=stream):
            got = g.linear_mx4(x, w, ws)
            back = g.dequantize_mx4(*g.quantize_mx4(x), columns=K)
    torch.cuda.synchronize()
    for i in range(3):
        x.mul_(-0.7 if i else 1.0)
        want, values = g.linear_mx4(x, w, ws), g.dequantize_mx4(*g.quantize_mx4(x))
        got.fill_(float("nan"))
        back.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(back, values), i


@pytest.mark.parametrize("M,N,K", [(1, 2048, 4096), (64, 64, 8192), (600, 520, 1024)])
def test_repeated_calls_give_the_same_bits(torch, M, N, K):
    a, sa = g.quantize_mx4(torch.randn(M, K, device="cuda"))
    b, sb = g.quantize_mx4(torch.randn(N, K, device="cuda"))
    want = g.matmul_mx4(a, sa, b, sb)
    for _ in range(3):
        assert torch.equal(g.matmul_mx4(a, sa, b, sb), want)


@pytest.mark.parametrize("M,N,K", [(4096, 8192, 16384), (4000, 7900, 14368)])
def test_large_products_with_scales_in_another_order(torch, M, N, K):
    """Shapes whose scales the plan puts in another order first, whole pairs of panels and in part."""
    d = g.gemm_mx4_plan_describe(M, N, K)
    assert d["workspace_bytes"] >= (M + N) * (K // 32), d
    torch.manual_seed(M)
    (a, sa), (b, sb) = ((torch.randint(0, 256, (r, K // 2), dtype=torch.uint8, device="cuda"),
                         torch.randint(126, 129, (r, K // 32), dtype=torch.uint8, device="cuda")) for r in (M, N))
    C = g.matmul_mx4(a, sa, b, sb)
    va, vb = (g.dequantize_mx4(q, s).double() for q, s in ((a, sa), (b, sb)))
    want = va @ vb.t().contiguous()
    bound = (K / 32) * 2.0 ** -23 * (va.abs() @ vb.abs().t().contiguous())       # a rounding to a block
    assert ((C.double() - want).abs() <= bound).all()
