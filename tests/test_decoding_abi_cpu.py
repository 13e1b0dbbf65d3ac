"""The C ABI of gemm_mx4.h and beam_search.h on a host without a GPU: every declared symbol is exported,
and bad arguments are refused before the HIP runtime is touched; the Python layer's checks."""
import ctypes
import os
import re

import pytest

import fp32_gemm_f32_amd as g
from test_ops_abi_cpu import ALIAS, ARG, DIM, LARGE, LD, P, PTR, ROOT, STEP, caller


@pytest.mark.parametrize("header,prefix", [("gemm_mx4.h", "gemm_mx4"), ("beam_search.h", "beam_step|reorder_beams")])
def test_exports_every_declared_symbol(header, prefix):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(rf"\b((?:{prefix})\w*)\s*\(", text))
    assert len(names) >= 3
    lib = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), f"{n} declared in {header} but not exported"


@pytest.mark.parametrize("back", [False, True])
def test_quantize_refusals(back):
    if back:
        call = caller("gemm_mx4_dequantize", "M K Q ldq s lds X t ldx stream",
                      (4, 40, P + STEP, 20, P + 2 * STEP, 2, P, 1, 40, None))
    else:
        call = caller("gemm_mx4_quantize", "M K X t ldx Q ldq s lds stream",
                      (4, 40, P, 1, 40, P + STEP, 20, P + 2 * STEP, 2, None))
    assert call(M=-1) == DIM and call(K=-1) == DIM
    assert call(ldx=39) == LD and call(ldq=19) == LD and call(lds=1) == LD and call(K=41, ldx=41) == LD
    assert call(K=0, ldq=0) == LD
    assert call(t=3) == ARG and call(t=-1) == ARG
    assert call(X=None) == PTR and call(Q=None) == PTR and call(s=None) == PTR
    assert call(X=P + 1) == PTR and call(t=0, X=P + 2) == PTR
    assert call(Q=P + 319) == ALIAS and call(s=P + 319) == ALIAS
    if not back:
        assert call(s=P + STEP + 79) == ALIAS
    assert call(M=0, X=None, Q=None, s=None) == 0 and call(K=0, X=None, Q=None, s=None) == 0


def test_product_refusals():
    call = caller("gemm_mx4", "M N K A lda sa ldsa B ldb sb ldsb bias C t ldc ws wsb stream",
                  (4, 4, 64, P, 32, P + STEP, 2, P + 2 * STEP, 32, P + 3 * STEP, 2, None, P + 4 * STEP, 0, 4,
                   None, 0, None))
    assert call(M=-1) == DIM and call(N=-1) == DIM and call(K=-2) == DIM and call(K=63) == DIM
    assert call(lda=31) == LD and call(ldb=31) == LD and call(ldsa=1) == LD and call(ldsb=1) == LD and call(ldc=3) == LD
    assert call(t=3) == ARG
    for name in ("A", "sa", "B", "sb", "C"):
        assert call(**{name: None}) == PTR, name
    assert call(C=P + 4 * STEP + 2) == PTR and call(bias=P + 5 * STEP + 2) == PTR
    assert call(wsb=64) == PTR and call(ws=P + 6 * STEP + 8, wsb=64) == PTR
    assert call(C=P + 124) == ALIAS and call(C=P + 2 * STEP) == ALIAS and call(C=P + STEP) == ALIAS
    assert call(C=P + 3 * STEP + 4) == ALIAS and call(bias=P + 4 * STEP + 60) == ALIAS
    assert call(ws=P + 4 * STEP, wsb=64) == ALIAS and call(ws=P, wsb=64) == ALIAS
    far = 1 << 40
    apart = dict(B=P + far, sa=P + 2 * far, sb=P + 3 * far, C=P + 4 * far)
    assert call(lda=1 << 23, **apart) == LARGE and call(ldsb=1 << 23, **apart) == LARGE
    assert call(M=1 << 30, N=1 << 10, ldc=1 << 10, A=P, B=P + (1 << 55), sa=P + (1 << 54), sb=P + (1 << 56),
                C=P + (1 << 50)) == LARGE
    assert call(M=0, A=None, C=None) == 0 and call(N=0, B=None, C=None) == 0


def test_plans_on_the_host():
    buf = ctypes.create_string_buffer(512)
    lib = g.library()
    assert lib.gemm_mx4_plan_describe(0, 4, 4, 256, buf, 512) == DIM
    assert lib.gemm_mx4_plan_describe(4, 4, 5, 256, buf, 512) == DIM
    assert lib.gemm_mx4_plan_describe(4, 4, 4, 256, None, 0) == ARG
    assert lib.gemm_mx4_plan_describe(4, 4, 4, 256, buf, 8) == ARG
    for M, N, K in [(1, 8192, 8192), (48, 16384, 4096), (1024, 1024, 1024), (8192, 8192, 8192), (17, 100, 16384)]:
        d = g.gemm_mx4_plan_describe(M, N, K, 256)
        assert d["splits"] >= 1 and d["workspace_bytes"] >= (d["splits"] > 1) * d["splits"] * M * N * 4


def test_step_refusals():
    call = caller("beam_step", "B W V x t ld s f pad top os ob ot ws wsb stream",
                  (2, 4, 100, P, 1, 100, P + STEP, None, 0, 4, P + 2 * STEP, P + 3 * STEP, P + 4 * STEP,
                   P + 5 * STEP, 1 << 15, None))
    assert call(B=-1) == DIM and call(W=-1) == DIM and call(V=-1) == DIM and call(V=0) == DIM
    assert call(ld=99) == LD
    assert call(t=5) == ARG and call(W=0) == ARG and call(W=65) == ARG and call(top=0) == ARG and call(top=65) == ARG
    for name in ("x", "s", "os", "ob", "ot"):
        assert call(**{name: None}) == PTR, name
    assert call(x=P + 1) == PTR and call(s=P + STEP + 2) == PTR and call(ob=P + 3 * STEP + 4) == PTR
    assert call(ws=P + 5 * STEP + 8) == PTR and call(ws=None) == PTR
    assert call(os=P + 1596) == ALIAS and call(ob=P + 2 * STEP + 16) == ALIAS and call(ot=P + STEP) == ALIAS
    assert call(f=P + 4 * STEP + 63) == ALIAS and call(ws=P + 3 * STEP) == ALIAS and call(ws=P + STEP - 16) == ALIAS
    assert call(B=0, x=None, s=None, os=None, ob=None, ot=None, ws=None, wsb=0) == 0
    assert g.beam_step_workspace_size(2, 65, 10, 0, 4) == 0 and g.beam_step_workspace_size(2, 4, 10, 3, 4) == 0


def test_reorder_refusals():
    # 6 rows of 4 pieces of 10 bytes, 64 apart; rows 1000 apart
    good = dict(src=P, dst=P + STEP, src_row=1000, dst_row=1000, count1=1, src_step1=0, dst_step1=0, count2=4,
                src_step2=64, dst_step2=64, run=10)

    def call(*states, B=2, W=3, beams=P + 8 * STEP, beam_bytes=8):
        try:
            g.reorder_beams_raw(B, W, beams, beam_bytes, [tuple({**good, **s}.values()) for s in states])
        except g.SgemmError as e:
            return e.status
        return 0
    assert call({}, B=-1) == DIM and call({}, W=-1) == DIM and call(dict(run=-1)) == DIM and call(dict(src_row=-8)) == DIM
    assert call(dict(dst_row=100)) == LD and call(dict(dst_step2=9)) == LD and call(dict(count1=2)) == LD
    assert call({}, beam_bytes=2) == ARG and call({}, W=65) == ARG
    assert call({}, beams=0) == PTR and call({}, beams=P + 8 * STEP + 4) == PTR
    assert call(dict(src=0)) == PTR and call(dict(dst=0)) == PTR
    assert call(dict(dst=P + 8 * STEP - 5000)) == ALIAS                     # beams
    assert call(dict(dst=P + 10)) == ALIAS and call(dict(dst=P, dst_row=1001)) == ALIAS
    assert call({}, {}) == ALIAS and call({}, dict(src=P + 2 * STEP)) == ALIAS
    assert call({}, dict(src=P + STEP + 100, dst=P + 3 * STEP)) == ALIAS    # reads what the first writes
    assert call(dict(dst=P + (1 << 60), count1=1 << 20, src_step1=1 << 20, dst_step1=1 << 20, count2=1 << 12,
                     src_step2=16, dst_step2=16, src_row=1 << 41, dst_row=1 << 41), beams=P - 64) == LARGE
    assert call({}, B=0) == 0 and call({}, W=0) == 0 and call() == 0
    assert call(dict(run=0, src=0, dst=0)) == 0


def test_python_layer_refusals():
    torch = pytest.importorskip("torch")
    q, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        g.quantize_mx4(torch.zeros(2, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        g.quantize_mx4(torch.zeros(2, 4))                    # not on a GPU
    with pytest.raises(TypeError):
        g.matmul_mx4(q.float(), s, q, s)
    with pytest.raises(ValueError):
        g.matmul_mx4(q, s, q, s)
    with pytest.raises(ValueError):
        g.dequantize_mx4(q, s)
    with pytest.raises(ValueError):
        g.linear_mx4(torch.zeros(2, 64), q, s)
    with pytest.raises(ValueError):
        g.beam_step(torch.zeros(2, 4), torch.zeros(1, 2))
    with pytest.raises(TypeError):
        g.beam_step(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        g.reorder_beams([torch.zeros(2, 4)], torch.zeros(1, 2, dtype=torch.int64))
