"""The 8-bit product and its quantiser against plain numpy in 64 bits, through the C ABI and
the tensor layer: odd sizes, strides and addresses, edge rows, the split form, other streams
and graph capture."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24                                  # half a step of FP32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
GUARD = 0x5b


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def codes(rng, rows, cols):
    return rng.integers(-128, 128, size=(rows, cols)).astype(np.int8)


def strided(torch, host, ld, offset, fill):
    """host in a GPU buffer of rows of ld elements after `offset` elements; the rest is
    `fill`."""
    rows, cols = host.shape
    buf = torch.full((offset + rows * ld + 1,), fill, dtype=host.dtype)
    view = buf[offset:offset + rows * ld].view(rows, ld)
    view[:, :cols] = host
    dev = buf.cuda()
    return dev, dev[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def guarded(torch, rows, cols, ld, dtype):
    """An output of rows x cols inside a buffer whose other bytes hold GUARD."""
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full(((rows + 2) * ld * size,), GUARD, dtype=torch.uint8, device="cuda")
    return raw, raw.view(dtype)[ld:(rows + 1) * ld].view(rows, ld)[:, :cols]


def assert_guard(raw, view, rows, cols, ld):
    size = view.element_size()
    b = raw.cpu().numpy().reshape(rows + 2, ld * size)
    assert (b[0] == GUARD).all() and (b[-1] == GUARD).all(), "wrote outside the rows"
    assert (b[1:-1, cols * size:] == GUARD).all(), "wrote past a row's end"


def reference(A, sa, B, sb, bias):
    total = A.astype(np.int64) @ B.astype(np.int64).T
    scaled = total.astype(np.float64) * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
    off = np.zeros(B.shape[0]) if bias is None else bias.astype(np.float64)
    return scaled, scaled + off[None, :], np.abs(scaled) + np.abs(off)[None, :]


def check(C, A, sa, B, sb, bias, out):
    """Roundings: the sum to FP32, the scales' product, the scaling, the bias: four of FP32
    on |scaled| + |bias|; then one of C's type (and its smallest step where C is subnormal)."""
    _, ref, size = reference(A, sa, B, sb, bias)
    tol = 4 * U32 * size
    tol = tol + HALF[out] * (np.abs(ref) + tol) + (2.0 ** -25 if out == "f16" else 0.0)
    got = C.float().cpu().numpy().astype(np.float64)
    worst = np.max(np.abs(got - ref) - tol) if got.size else -1
    assert worst <= 0, f"off by {worst} more than the roundings"


SHAPES = [(1, 1, 1), (1, 64, 16), (1, 1000, 4096), (2, 3, 5), (3, 129, 127), (7, 65, 300),
          (16, 257, 1024), (17, 96, 640), (33, 1024, 8192), (48, 500, 4096), (64, 64, 131056),
          (65, 66, 67), (100, 300, 129), (128, 128, 128), (130, 260, 1040), (255, 257, 513),
          (256, 256, 384), (300, 1, 2000), (513, 511, 1000), (1000, 700, 528), (640, 1100, 1025),
          (2100, 2050, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_product(torch, M, N, K, out):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    A, B = codes(rng, M, K), codes(rng, N, K)
    sa = rng.uniform(1e-4, 1e-2, M).astype(np.float32)
    sb = rng.uniform(1e-4, 1e-2, N).astype(np.float32)
    bias = rng.standard_normal(N).astype(np.float32) if (M + N) % 2 else None
    _, dA = strided(torch, torch.from_numpy(A), K, 0, 99)
    _, dB = strided(torch, torch.from_numpy(B), K, 0, -77)
    raw, C = guarded(torch, M, N, N + 3, dtype_of(torch, out))
    print(f"[i8] {M}x{N}x{K} {out}", flush=True)
    g.matmul_i8(dA, torch.from_numpy(sa).cuda(), dB, torch.from_numpy(sb).cuda(),
                bias=None if bias is None else torch.from_numpy(bias).cuda(), out=C)
    torch.cuda.synchronize()
    check(C, A, sa, B, sb, bias, out)
    assert_guard(raw, C, M, N, N + 3)


TILES = [("i8_64x32", "aligned", 8763, 65, 704), ("i8_64x32", "any", 18, 68, 655),
         ("i8_64x64", "aligned", 18, 66, 672), ("i8_64x64", "any", 18, 8484, 857),
         ("i8_64x128", "any", 8319, 68, 922),
         ("i8_64x128_w8", "aligned", 65, 8333, 672), ("i8_64x128_w8", "any", 68, 8193, 726),
         ("i8_128x128", "aligned", 715, 2733, 640),
         ("i8_128x128_s4", "aligned", 193, 8855, 720), ("i8_128x128_s4", "any", 194, 8427, 707),
         ("i8_192x128", "any", 5451, 644, 655), ("i8_128x256", "aligned", 8457, 414, 656),
         ("i8_192x256", "aligned", 1040, 7235, 704), ("i8_192x256", "any", 8371, 777, 705),
         ("i8_256x256", "aligned", 3356, 2315, 640), ("i8_256x256", "any", 6967, 1557, 644),
         # more tiles than compute units: workgroups go on to another one, or two; the last
         # K has as many panels as stages, then fewer
         ("i8_128x128_s4", "aligned", 6740, 1028, 2976), ("i8_128x256", "aligned", 2070, 7361, 912),
         ("i8_192x256", "aligned", 2983, 10898, 416), ("i8_256x256", "aligned", 3500, 5803, 272),
         ("i8_256x256", "aligned", 2565, 14022, 144), ("i8_256x256", "aligned", 7281, 2842, 128)]


@pytest.mark.parametrize("name,form,M,N,K", TILES)
def test_every_tile(torch, name, form, M, N, K):
    """A product for each tile of the plan (at 256 compute units), with edges in both
    directions and a ring of panels that turns over."""
    d = g.gemm_i8_plan_describe(M, N, K, num_cus=256)
    assert (d["name"], d["form"], d["copies"]) == (name, form, [False, False])
    rng = np.random.default_rng(M + N + K)
    A, B = codes(rng, M, K), codes(rng, N, K)
    sa = rng.uniform(1e-4, 1e-2, M).astype(np.float32)
    sb = rng.uniform(1e-4, 1e-2, N).astype(np.float32)
    bias = rng.standard_normal(N).astype(np.float32)
    dA, dB = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    dsa, dsb, dbias = (torch.from_numpy(x).cuda() for x in (sa, sb, bias))
    raw, C = guarded(torch, M, N, N + 1, torch.float32)
    print(f"[i8] {name} {form} {M}x{N}x{K}", flush=True)
    g.matmul_i8(dA, dsa, dB, dsb, bias=dbias, out=C)
    torch.cuda.synchronize()
    # sums of K products stay far below 2^53: exact in 64-bit floats
    scaled = (A.astype(np.float64) @ B.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sb
    ref = scaled + bias
    tol = 4 * U32 * (np.abs(scaled) + np.abs(bias)) + U32 * np.abs(ref) * (1 + 4 * U32)
    worst = np.max(np.abs(C.cpu().numpy() - ref) - tol)
    assert worst <= 0, f"off by {worst} more than the roundings"
    assert_guard(raw, C, M, N, N + 1)


@pytest.mark.parametrize("M,N,K,lda,ldb,ao,bo", [
    (70, 90, 256, 272, 260, 0, 0),        # aligned rows with padding: the direct loads
    (70, 90, 256, 257, 259, 0, 0),        # odd strides
    (70, 90, 256, 256, 256, 1, 3),        # odd addresses
    (5, 333, 200, 203, 201, 2, 5),        # few rows
    (1, 777, 1234, 1234, 1235, 1, 1),
    (1, 512, 1024, 1024, 1040, 0, 4),
    (300, 280, 144, 148, 160, 4, 8),
])
def test_strides_and_addresses(torch, M, N, K, lda, ldb, ao, bo):
    rng = np.random.default_rng(lda + ldb)
    A, B = codes(rng, M, K), codes(rng, N, K)
    one = np.float32(1.0)
    keep_a, dA = strided(torch, torch.from_numpy(A), lda, ao, 99)
    keep_b, dB = strided(torch, torch.from_numpy(B), ldb, bo, -77)
    print(f"[i8] {M}x{N}x{K} ld {lda} {ldb} offsets {ao} {bo}", flush=True)
    C = g.matmul_i8(dA, torch.ones(M, device="cuda"), dB, torch.ones(N, device="cuda"))
    # unit scales: the sum itself, rounded once
    want = (A.astype(np.int64) @ B.astype(np.int64).T).astype(np.float32)
    assert np.array_equal(C.cpu().numpy(), want * one)


def test_extreme_values_do_not_overflow(torch):
    K = 131071
    for a, b in [(-128, -128), (-128, 127), (127, 127)]:
        A = torch.full((2, K), a, dtype=torch.int8, device="cuda")
        B = torch.full((3, K), b, dtype=torch.int8, device="cuda")
        C = g.matmul_i8(A, torch.ones(2, device="cuda"), B, torch.ones(3, device="cuda"))
        assert (C.cpu().numpy() == np.float32(a * b * K)).all(), (a, b)


def test_special_scales(torch):
    """NaN and infinite scales follow the formula, in their own rows and columns only."""
    rng = np.random.default_rng(5)
    A, B = codes(rng, 40, 64), codes(rng, 50, 64)
    sa, sb = np.ones(40, np.float32), np.ones(50, np.float32)
    sa[3], sa[7], sa[9], sb[11] = np.nan, np.inf, 0.0, -2.0
    C = g.matmul_i8(torch.from_numpy(A).cuda(), torch.from_numpy(sa).cuda(),
                    torch.from_numpy(B).cuda(), torch.from_numpy(sb).cuda()).cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = (A.astype(np.int64) @ B.astype(np.int64).T).astype(np.float32) * (sa[:, None] * sb[None, :])
    np.testing.assert_array_equal(C, want)


def test_empty_shapes(torch):
    z = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda n: torch.full((n,), float("nan"), device="cuda")      # noqa: E731
    assert g.matmul_i8(z(0, 8), f(0), z(4, 8), f(4)).shape == (0, 4)
    assert g.matmul_i8(z(4, 8), f(4), z(0, 8), f(0)).shape == (4, 0)
    bias = torch.arange(5, dtype=torch.float32, device="cuda")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        C = g.matmul_i8(z(3, 0), f(3), z(5, 0), f(5), bias=bias, out_dtype=dt)
        assert torch.equal(C.float(), bias.expand(3, 5))
    assert (g.matmul_i8(z(3, 0), f(3), z(5, 0), f(5)) == 0).all()


@pytest.mark.parametrize("M,N,K", [(96, 80, 16384), (9, 70, 65536), (700, 690, 8000), (1030, 1100, 1027),
                                   (300, 5000, 4095), (24, 48, 20001)])
def test_with_and_without_workspace(torch, M, N, K):
    """The forms that use a workspace (split, copied into place) and those that run without
    give the same bits; a workspace that is too small is refused."""
    size = g.gemm_i8_workspace_size(M, N, K)
    assert size > 0 or K < 10000          # a long K over few tiles is split
    rng = np.random.default_rng(8)
    A, B = torch.from_numpy(codes(rng, M, K)).cuda(), torch.from_numpy(codes(rng, N, K)).cuda()
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    C = g.matmul_i8(A, sa, B, sb, out_dtype=torch.bfloat16)
    D = torch.empty_like(C)
    args = (M, N, K, A.data_ptr(), K, sa.data_ptr(), B.data_ptr(), K, sb.data_ptr(), 0,
            D.data_ptr(), 1, N)
    g.gemm_i8(*args, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(C, D)
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    if size > 64:
        with pytest.raises(g.SgemmError) as e:
            g.gemm_i8(*args, ws.data_ptr(), 64)
        assert e.value.status == -6


@pytest.mark.parametrize("M,N,K", [(17, 40, 200), (64, 96, 384), (130, 70, 1000), (260, 300, 513),
                                   (1500, 2100, 130), (2300, 2500, 257), (4200, 4100, 40)])
@pytest.mark.parametrize("lda,ldb,ao,bo", [(0, 0, 0, 0), (1, 2, 1, 0), (3, 5, 2, 3), (0, 4, 3, 1)])
def test_rows_of_any_alignment_without_workspace(torch, M, N, K, lda, ldb, ao, bo):
    """Rows at every offset from a word's boundary and every remainder of K, in the tiles' own
    loads (no workspace, so nothing is copied into place first). The buffers end with the
    matrices' last byte."""
    rng = np.random.default_rng(M + K + lda)
    A, B = codes(rng, M, K), codes(rng, N, K)

    def flush(host, ld, offset):
        rows = host.shape[0]
        dev = torch.full((offset + (rows - 1) * ld + K,), -128, dtype=torch.int8, device="cuda")
        dev.as_strided((rows, K), (ld, 1), offset).copy_(torch.from_numpy(host))
        return dev, dev.data_ptr() + offset
    for k in (K, K - 1, K - 2, K - 3):
        keep_a, pa = flush(A, K + lda, ao)
        keep_b, pb = flush(B, K + ldb, bo)
        C = torch.empty(M, N, device="cuda")
        one = torch.ones(max(M, N), device="cuda")
        print(f"[i8 any] {M}x{N}x{k} ld +{lda} +{ldb} offsets {ao} {bo}", flush=True)
        g.gemm_i8(M, N, k, pa, K + lda, one.data_ptr(), pb, K + ldb, one.data_ptr(), 0,
                  C.data_ptr(), 0, N, stream=torch.cuda.current_stream().cuda_stream)
        want = (A[:, :k].astype(np.float64) @ B[:, :k].astype(np.float64).T).astype(np.float32)
        assert np.array_equal(C.cpu().numpy(), want)


def quantized(x):
    """The definition in FP32, row by row (numpy divides and multiplies with one rounding)."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        peak = np.max(np.abs(x), axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
        scale, inverse = peak / np.float32(127), np.float32(127) / peak
        dead = np.isinf(inverse)
        scale = np.where(dead, np.float32(0), scale)
        q = np.rint(x * inverse[:, None])
        q = np.where(dead[:, None] | np.isnan(q), 0, np.clip(q, -127, 127)).astype(np.int8)
    return q, scale


@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (3, 64), (5, 100), (2, 1000), (17, 2048),
                                 (4, 4097), (3, 8192), (300, 515), (2, 20011), (1, 70000),
                                 (2000, 33), (5, 0), (70, 64),
                                 (33, 127), (65, 255), (130, 512), (9, 1030), (600, 9000), (520, 16383)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_quantize(torch, M, K, dt, pad, offset):
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy((rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))))
                         .astype(np.float32)).to(dtype_of(torch, dt))
    keep, dX = strided(torch, x, K + pad, offset, float("nan"))
    ldq = K + pad + 2
    raw, Q = guarded(torch, M, K, ldq, torch.int8)
    print(f"[quantize] {M}x{K} {dt} pad {pad}", flush=True)
    _, scales = g.quantize_rows(dX, out=Q)
    q, s = quantized(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(Q.cpu().numpy(), q)
    assert_guard(raw, Q, M, K, ldq)


@pytest.mark.parametrize("K", [9, 520, 9001])
def test_quantize_edge_rows(torch, K):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((10, K)).astype(np.float32)
    x[0] = 0.0
    x[1] = 1e-39                                   # 127 / peak overflows
    x[2, K - 1] = np.nan
    x[3, 0] = -np.inf
    x[4, 1], x[4, K - 2] = np.inf, np.nan
    x[5] = np.float32(3.4e38)
    x[6] = -x[6].max() * np.float32(2)             # one value throughout: -127
    x[7] = np.arange(K) % 255 - 127                # halves on a scale of 1
    x[7, 3:] += 0.5
    x[7, 0], x[7, 1], x[7, 2] = 127, -127, 0.5
    x[7] = np.clip(x[7], -127, 127)
    x[8] = -0.0
    x[9] = 4e-37
    Q, scales = g.quantize_rows(torch.from_numpy(x).cuda())
    q, s = quantized(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    assert np.isnan(s[2]) and np.isinf(s[3]) and np.isnan(s[4]) and s[0] == s[1] == 0


def test_quantize_empty(torch):
    Q, s = g.quantize_rows(torch.empty(0, 5, device="cuda"))
    assert Q.shape == (0, 5) and s.shape == (0,)


def test_linear(torch):
    """Quantising and multiplying come within the quantisation's error of the FP32 product:
    each operand is off by at most half a step of its scale."""
    rng = np.random.default_rng(3)
    X, W = rng.standard_normal((2, 19, 512)).astype(np.float32), rng.standard_normal((77, 512)).astype(np.float32)
    wq, ws = g.quantize_rows(torch.from_numpy(W).cuda())
    Y = g.linear_i8(torch.from_numpy(X).cuda(), wq, ws)
    assert Y.shape == (2, 19, 77) and Y.dtype == torch.float32
    x = X.reshape(-1, 512).astype(np.float64)
    w = W.astype(np.float64)
    hx = np.abs(x).max(1, keepdims=True) / 254 * (1 + 2.0 ** -10)
    hw = np.abs(w).max(1, keepdims=True) / 254 * (1 + 2.0 ** -10)
    bound = np.abs(x).sum(1, keepdims=True) * hw.T + hx * np.abs(w).sum(1)[None, :] + 512 * hx * hw.T
    assert (np.abs(Y.cpu().numpy().reshape(-1, 77) - x @ w.T) <= bound + 1e-4).all()


def test_other_layouts(torch):
    """Transposed and broadcast inputs are copied, not misread; bad shapes are refused."""
    rng = np.random.default_rng(4)
    A, B = codes(rng, 24, 48), codes(rng, 40, 48)
    dAt, dBt = torch.from_numpy(A.T.copy()).cuda().t(), torch.from_numpy(B.T.copy()).cuda().t()
    one = torch.ones(1, device="cuda")
    C = g.matmul_i8(dAt, one.expand(24), dBt, one.expand(40))
    assert np.array_equal(C.cpu().numpy(), (A.astype(np.int64) @ B.astype(np.int64).T).astype(np.float32))
    row = torch.randn(1, 100, device="cuda").expand(6, 100)
    q, s = g.quantize_rows(row)
    q1, s1 = g.quantize_rows(row[:1])
    assert torch.equal(q, q1.expand(6, 100)) and torch.equal(s, s1.expand(6))
    with pytest.raises(ValueError):
        g.matmul_i8(dAt, one.expand(23), dBt, one.expand(40))
    with pytest.raises(TypeError):
        g.matmul_i8(dAt, one.expand(24).double(), dBt, one.expand(40))
    with pytest.raises(ValueError):
        g.matmul_i8(dAt, one.expand(24), dBt[:, 1:], one.expand(40))
    with pytest.raises(ValueError):
        g.matmul_i8(dAt, one.expand(24), dBt, one.expand(40), out=torch.empty(24, 41, device="cuda"))
    with pytest.raises(g.SgemmError) as e:
        big = torch.zeros(1, 131072, dtype=torch.int8, device="cuda")
        g.matmul_i8(big, one, big, one)
    assert e.value.status == -7


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (96, 80, 16384), (300, 280, 528), (65, 66, 67)])
def test_graph_capture_and_other_stream(torch, M, N, K):
    rng = np.random.default_rng(K)
    x = torch.randn(M, K, device="cuda")
    B = torch.from_numpy(codes(rng, N, K)).cuda()
    sb = torch.rand(N, device="cuda")
    want = g.linear_i8(x, B, sb)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    print(f"[i8 graph] {M}x{N}x{K}", flush=True)
    with torch.cuda.stream(stream):
        assert torch.equal(g.linear_i8(x, B, sb), want)
        with torch.cuda.graph(graph, stream=stream):
            got = g.linear_i8(x, B, sb)
    torch.cuda.synchronize()
    for i in range(3):
        x.mul_(-0.5 if i else 1.0)
        want = g.linear_i8(x, B, sb)               # eager work between the replays
        got.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
