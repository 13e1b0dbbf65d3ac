"""The operators of decoding over more rows than one launch takes: every row is served, on both sides of
a launch's border."""
import pytest

import fp32_gemm_f32_amd as g
from test_gpu_many_rows import ITEMS, windows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    yield t
    t.cuda.empty_cache()


def test_quantize_and_back(torch):
    K = 2
    border = (2 ** 31 - 1024) // 4                 # rows of four units, fewer than 2^31 units
    M = border + 1029
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.full((M, 1), 0x77, dtype=torch.uint8, device="cuda")
    s = torch.full((M, 1), 0x77, dtype=torch.uint8, device="cuda")
    print(f"[many rows] mx4 quantize {M}x{K}", flush=True)
    g.quantize_mx4(x, out=q, scales=s)
    for w in windows(border, M):
        a, b = g.quantize_mx4(x[w].clone())
        assert torch.equal(q[w], a) and torch.equal(s[w], b)
    del x
    y = torch.full((M, K), 99.0, dtype=torch.bfloat16, device="cuda")
    g.dequantize_mx4(q, s, out=y)
    for w in windows(border, M):
        assert torch.equal(y[w], g.dequantize_mx4(q[w].clone(), s[w].clone(), dtype=torch.bfloat16))


def test_beam_step(torch):
    border = ITEMS // 256
    B, V = border + 1029, 3
    x = torch.empty(B, V, dtype=torch.float16, device="cuda").normal_()
    scores = torch.zeros(B, 1, device="cuda")
    print(f"[many rows] beams {B}x1x{V}", flush=True)
    r = g.beam_step(x, scores, top=2)
    for w in windows(border, B):
        part = g.beam_step(x[w].clone(), scores[w].clone(), top=2)
        assert torch.equal(r.beams[w], part.beams) and torch.equal(r.tokens[w], part.tokens)
        # rows at other addresses: their three terms may be added in another order, eight roundings of at
        # most 2^-22 (totals stay below 8)
        assert (r.scores[w] - part.scores).abs().max() <= 8 * 2.0 ** -22
        best = x[w].float().sort(dim=1, descending=True, stable=True)
        assert torch.equal(r.tokens[w], best.indices[:, :2])


def test_reorder(torch):
    border = ITEMS // 256                          # requests, a workgroup each
    B = border + 1029
    t = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1).repeat(1, 2).view(2 * B, 1)
    t[1::2] += 7
    beams = torch.randint(0, 2, (B, 2), device="cuda", dtype=torch.int32)
    print(f"[many rows] reorder {B}x2", flush=True)
    out = g.reorder_beams([t], beams)[0].view(B, 2)
    for w in windows(border, B):
        want = torch.arange(B, dtype=torch.int32, device="cuda")[w][:, None] + 7 * beams[w]
        assert torch.equal(out[w], want)


def test_the_longest_row(torch):
    """2^31 - 1 elements: a unit of eight starts at 2^31 - 8 and ends past what 31 bits count."""
    K = 2 ** 31 - 1
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    end = torch.randn(1, 33, device="cuda").bfloat16()
    x[:, -31:] = end[:, :31]                       # the last block, 31 of 32
    x[:, :32] = end[:, :32]
    print(f"[many rows] mx4 quantize 1x{K}", flush=True)
    q = torch.full((1, 2 ** 30 + 16), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 2 ** 26 + 16), 0x55, dtype=torch.uint8, device="cuda")
    g.quantize_mx4(x, out=q[:, :2 ** 30], scales=s[:, :2 ** 26])
    for part, at in [(end[:, :31], 2 ** 31 - 32), (end[:, :32], 0)]:
        a, b = g.quantize_mx4(part.contiguous())
        assert torch.equal(q[:, at // 2:at // 2 + 16], a) and torch.equal(s[:, at // 32:at // 32 + 1], b)
    assert not q[:, 16:2 ** 30 - 16].any() and not s[:, 1:2 ** 26 - 1].any()
    assert (q[:, 2 ** 30:] == 0x55).all() and (s[:, 2 ** 26:] == 0x55).all()
    y = torch.full((1, 2 ** 31 + 31), 9.0, dtype=torch.bfloat16, device="cuda")
    g.dequantize_mx4(q[:, :2 ** 30], s[:, :2 ** 26], columns=K, out=y[:, :K])
    a, b = g.quantize_mx4(end[:, :31].contiguous())
    assert torch.equal(y[:, K - 31:K], g.dequantize_mx4(a, b, dtype=torch.bfloat16, columns=31))
    assert not y[:, 32:K - 31].any() and (y[:, K:] == 9.0).all()
    del x, y
    with pytest.raises(ValueError):                # 2^31 elements
        g.dequantize_mx4(q[:, :2 ** 30], s[:, :2 ** 26])
    with pytest.raises(ValueError):
        g.matmul_mx4(q[:, :2 ** 30], s[:, :2 ** 26], q[:, :2 ** 30], s[:, :2 ** 26])
