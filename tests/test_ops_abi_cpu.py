"""The C ABI of gemm_i8.h and token_logprobs.h on a host without a GPU: every declared symbol
is exported, and bad arguments are refused before the HIP runtime is touched. The Python
layer's checks of types and shapes are here too."""
import ctypes
import os
import re

import pytest

import fp32_gemm_f32_amd as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DIM, LD, PTR, ALIAS, ARG, LARGE = -1, -2, -3, -4, -6, -7
P = 1 << 20         # fake, 16-byte aligned "device" addresses: never dereferenced here
STEP = 1 << 16


@pytest.mark.parametrize("header", ["gemm_i8.h", "token_logprobs.h"])
def test_exports_every_declared_symbol(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b((?:gemm_i8|token_logprobs)\w*)\s*\(", text))
    assert len(names) >= 3
    lib = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), f"{n} declared in {header} but not exported"


def caller(fn, names, ok):
    names = names.split()
    assert len(names) == len(ok)

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return getattr(g.library(), fn)(*args)
    return call


def test_quantize_rows_refusals():
    call = caller("gemm_i8_quantize_rows", "M K X t ldx Q ldq s stream",
                  (4, 8, P, 1, 8, P + STEP, 8, P + 2 * STEP, None))
    assert call(M=-1) == DIM and call(K=-1) == DIM
    assert call(ldx=7) == LD and call(ldq=7) == LD and call(K=0, ldx=0) == LD
    assert call(t=3) == ARG and call(t=-1) == ARG
    assert call(X=None) == PTR and call(Q=None) == PTR and call(s=None) == PTR
    assert call(X=P + 1) == PTR and call(t=0, X=P + 2) == PTR and call(s=P + 2 * STEP + 2) == PTR
    assert call(Q=P + 63) == ALIAS and call(s=P + 60) == ALIAS and call(s=P + STEP + 28) == ALIAS
    assert call(M=0, X=None, Q=None, s=None) == 0


def test_gemm_i8_refusals():
    call = caller("gemm_i8", "M N K A lda sa B ldb sb bias C t ldc ws wsb stream",
                  (4, 4, 8, P, 8, P + STEP, P + 2 * STEP, 8, P + 3 * STEP, None, P + 4 * STEP, 0, 4,
                   None, 0, None))
    assert call(M=-1) == DIM and call(N=-1) == DIM and call(K=-1) == DIM
    assert call(lda=7) == LD and call(ldb=7) == LD and call(ldc=3) == LD
    assert call(t=3) == ARG
    for name in ("A", "sa", "B", "sb", "C"):
        assert call(**{name: None}) == PTR, name
    assert call(sa=P + STEP + 1) == PTR and call(C=P + 4 * STEP + 2) == PTR
    assert call(bias=P + 5 * STEP + 2) == PTR
    assert call(t=1, C=P + 4 * STEP + 1) == PTR
    assert call(wsb=64) == PTR and call(ws=P + 6 * STEP + 8, wsb=64) == PTR
    assert call(C=P + 28) == ALIAS and call(C=P + 2 * STEP) == ALIAS
    assert call(C=P + STEP) == ALIAS and call(bias=P + 4 * STEP + 60) == ALIAS
    assert call(ws=P + 4 * STEP, wsb=64) == ALIAS and call(ws=P, wsb=64) == ALIAS
    far = 1 << 40
    assert call(K=131072, lda=131072, ldb=131072, B=P + far, sa=P + 2 * far, sb=P + 3 * far,
                C=P + 4 * far) == LARGE
    assert call(lda=1 << 23, B=P + far, sa=P + 2 * far, sb=P + 3 * far, C=P + 4 * far) == LARGE
    assert call(M=0, A=None, C=None) == 0 and call(N=0, B=None, C=None) == 0


def test_gemm_i8_plan_on_the_host():
    buf = ctypes.create_string_buffer(512)
    lib = g.library()
    assert lib.gemm_i8_plan_describe(0, 4, 4, 4, 4, 256, buf, 512) == DIM
    assert lib.gemm_i8_plan_describe(4, 4, 4, 3, 4, 256, buf, 512) == LD
    assert lib.gemm_i8_plan_describe(4, 4, 4, 4, 4, 256, None, 0) == ARG
    assert lib.gemm_i8_plan_describe(4, 4, 4, 4, 4, 256, buf, 8) == ARG
    assert lib.gemm_i8_plan_describe(4, 4, 131072, 131072, 131072, 256, buf, 512) == LARGE
    seen = set()
    for M, N, K in [(1, 1, 1), (1, 64, 64), (1, 8192, 8192), (16, 64, 131071), (48, 16384, 4096),
                    (1024, 1024, 1024), (1023, 1025, 1027), (8192, 8192, 8192), (64, 64, 131071),
                    (65, 130, 16384), (100000, 1, 1), (4096, 4096, 4096), (1024, 4096, 4096),
                    (2000, 16000, 500), (128, 8192, 8192), (1024, 4096, 8192), (2048, 2048, 2048)]:
        for pad_a, pad_b in [(0, 0), (5, 0), (0, 3), (13, 13), (16, 4)]:
            d = g.gemm_i8_plan_describe(M, N, K, K + pad_a, K + pad_b, num_cus=256)
            seen.add(d["name"])
            assert d["tiles"][0] * d["BM"] >= M > (d["tiles"][0] - 1) * d["BM"]
            assert d["tiles"][1] * d["BN"] >= N > (d["tiles"][1] - 1) * d["BN"]
            # the splits cover K, none of them empty, and start on whole panels
            assert d["splits"] * d["k_chunk"] >= K > (d["splits"] - 1) * d["k_chunk"]
            assert d["splits"] == 1 or d["k_chunk"] % 128 == 0
            k16 = (K + 15) // 16 * 16
            want = (d["splits"] * M * N * 4 + 15) // 16 * 16 if d["splits"] > 1 else 0
            want += (M * k16 if d["copies"][0] else 0) + (N * k16 if d["copies"][1] else 0)
            assert d["workspace_bytes"] == want
            # the aligned form only ever sees rows it can load
            fit = [K % 16 == 0 and p % 4 == 0 for p in (pad_a, pad_b)]
            if d["form"] == "aligned":
                assert all(f or c for f, c in zip(fit, d["copies"]))
            assert not any(f and c for f, c in zip(fit, d["copies"]))
    assert len(seen) >= 5, seen


def test_token_logprobs_refusals():
    call = caller("token_logprobs", "M V x t ld tok tb lp ent lse top tv ti ws wsb stream",
                  (4, 100, P, 1, 100, P + STEP, 8, P + 2 * STEP, P + 3 * STEP, P + 4 * STEP, 2,
                   P + 5 * STEP, P + 6 * STEP, None, 0, None))
    assert call(M=-1) == DIM and call(V=-1) == DIM and call(V=0) == DIM
    assert call(ld=99) == LD
    assert call(t=9) == ARG and call(tb=2) == ARG and call(top=65) == ARG and call(top=-1) == ARG
    assert call(V=1) == ARG                                  # top > V
    for name in ("x", "tok", "lp", "tv", "ti"):
        assert call(**{name: None}) == PTR, name
    assert call(x=P + 1) == PTR and call(tok=P + STEP + 4) == PTR and call(ti=P + 6 * STEP + 4) == PTR
    assert call(ws=P + 7 * STEP + 4, wsb=64) == PTR and call(wsb=64) == PTR
    assert call(lp=P + 796) == ALIAS and call(lse=P + 3 * STEP + 12) == ALIAS
    assert call(lp=P + STEP) == ALIAS and call(ws=P, wsb=64) == ALIAS
    assert call(ws=P + 5 * STEP, wsb=16) == ALIAS
    assert call(M=0, x=None, tok=None, lp=None, tv=None, ti=None) == 0


def test_token_logprobs_backward_refusals():
    call = caller("token_logprobs_backward",
                  "M V x t ld tok tb lse ent glp gent glse dx ldg stream",
                  (4, 100, P, 1, 100, P + STEP, 8, P + 2 * STEP, P + 3 * STEP, P + 4 * STEP,
                   P + 5 * STEP, P + 6 * STEP, P + 7 * STEP, 100, None))
    assert call(M=-1) == DIM and call(V=0) == DIM
    assert call(ld=99) == LD and call(ldg=99) == LD
    assert call(t=3) == ARG and call(tb=0) == ARG
    for name in ("x", "tok", "lse", "ent", "dx"):
        assert call(**{name: None}) == PTR, name
    assert call(glp=P + 4 * STEP + 1) == PTR and call(dx=P + 7 * STEP + 1) == PTR
    assert call(dx=P + 2) == ALIAS and call(dx=P, ldg=101) == ALIAS
    assert call(dx=P + 2 * STEP) == ALIAS and call(dx=P + 6 * STEP) == ALIAS
    assert call(M=0, x=None, tok=None, lse=None, ent=None, dx=None) == 0


def test_workspace_sizes_of_refused_shapes():
    assert g.gemm_i8_workspace_size(-1, 4, 4) == 0 and g.gemm_i8_workspace_size(4, 4, 131072) == 0
    assert g.gemm_i8_workspace_size(4, 4, 8, P, 7, P, 8) == 0
    assert g.token_logprobs_workspace_size(4, 100, 7, 0) == 0
    assert g.token_logprobs_workspace_size(4, 100, 0, 101) == 0


def test_python_layer_refusals():
    torch = pytest.importorskip("torch")
    i8, f = torch.zeros(2, 4, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(TypeError):
        g.quantize_rows(torch.zeros(2, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        g.quantize_rows(torch.zeros(2, 4))                   # not on a GPU
    with pytest.raises(TypeError):
        g.matmul_i8(torch.zeros(2, 4), f, i8, f)
    with pytest.raises(ValueError):
        g.matmul_i8(i8, f, i8, f)
    with pytest.raises(TypeError):
        g.token_logprobs(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        g.token_logprobs(torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64))
