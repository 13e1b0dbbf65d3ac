"""Python binding of the MI355X FP32 GEMM library (libsgemm_f32.so).

Argument marshalling only: every call goes straight to the C ABI of include/sgemm_f32.h,
and every step of the product runs in the library's HIP kernels. There is no fallback:
if the library is not built, importing the binding's functions raises.

Raw layer (same names and arguments as the C ABI; pointers are integers):
    sgemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=0)
    sgemm_f32_naive(...), sgemm_f32_tiled(..., tile=32, pad=0, stream=0)
    sgemm_f32_splitk(..., splits, workspace, workspace_bytes, stream=0)
    sgemm_f32_splitk_workspace_size(M, N, K, splits) -> int
    sgemm_f32_streamk(..., variant, workspace, workspace_bytes, stream=0)
    sgemm_f32_streamk_workspace_size(M, N, K, lda, ldb, ldc, variant=-1) -> int
    sgemm_f32_streamk_noalloc(..., variant, stream=0)
    sgemm_f32_streamk_noalloc_scratch_bytes() -> int
    sgemm_f32_streamk_describe(M, N, K, variant=-1, num_cus=0) -> dict
    sgemm_f32_regtiled(..., tm=4, tn=4, stream=0)
    sgemm_f32_lds_transpose(rows, cols, src, ldi, dst, ldo, tile=32, pad=0, stream=0)
    sgemm_f32_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=0)
    sgemm_f32_plan_describe(M, N, K, A, lda, B, ldb, C, ldc, num_cus=0) -> dict
    sgemm_f32_variant_describe(variant, M, N, K, lda, ldb, ldc, num_cus=0) -> dict
    sgemm_f32_variant_info(variant) -> dict, planned_variants() -> [index],
    streamk_variants() -> [index]
    gemm_i8_quantize_rows(M, K, X, x_dtype, ldx, Q, ldq, scales, stream=0)
    gemm_i8(M, N, K, A, lda, a_scales, B, ldb, b_scales, bias, C, c_dtype, ldc,
            workspace=0, workspace_bytes=0, stream=0)
    gemm_i8_workspace_size(M, N, K, A=0, lda=K, B=0, ldb=K) -> int
    gemm_i8_plan_describe(M, N, K, lda=K, ldb=K, num_cus=0) -> dict
    token_logprobs_raw(...), token_logprobs_workspace_size(M, V, dtype, top) -> int,
    token_logprobs_backward_raw(...): token_logprobs.h's arguments in their order, lse_low (of the
    forms that have it) by name
    gemm_mx4_quantize(M, K, X, x_dtype, ldx, Q, ldq, scales, lds, stream=0)
    gemm_mx4_dequantize(M, K, Q, ldq, scales, lds, Y, y_dtype, ldy, stream=0)
    gemm_mx4(M, N, K, A, lda, a_scales, lda_scales, B, ldb, b_scales, ldb_scales, bias, C, c_dtype,
             ldc, workspace=0, workspace_bytes=0, stream=0)
    gemm_mx4_workspace_size(M, N, K, A=0, lda=.., a_scales=0, .., B=0, .., b_scales=0, ..) -> int
    gemm_mx4_plan_describe(M, N, K, num_cus=0) -> dict
    beam_step_raw(...), beam_step_workspace_size(B, W, V, dtype, top) -> int,
    reorder_beams_raw(B, W, beams, beam_bytes, states, stream=0): beam_search.h's arguments in their
    order, a state a tuple of beam_state's fields
Tensor layer (torch tensors on the GPU, launched on torch's current stream):
    matmul(A, B, out=None, kernel="auto", variant=-1) -> C
    quantize_rows(X, out=None, scales=None) -> (Q, scales)
    matmul_i8(A, a_scales, B, b_scales, bias=None, out_dtype=None, out=None) -> C
    linear_i8(X, B, b_scales, bias=None, out_dtype=None) -> C
    token_logprobs(logits, tokens, top=0) -> TokenLogprobs (differentiable in logits)
    token_logprobs_backward(logits, tokens, lse, entropy, grad_logprobs, grad_entropy=None,
                            grad_lse=None, out=None, lse_low=None) -> gradient of the logits
    quantize_mx4(X, out=None, scales=None) -> (Q, scales)
    dequantize_mx4(Q, scales, dtype=None, columns=None, out=None) -> values
    matmul_mx4(A, a_scales, B, b_scales, bias=None, out_dtype=None, out=None) -> C
    linear_mx4(X, B, b_scales, bias=None, out_dtype=None) -> C
    beam_step(logits, scores, top=None, finished=None, pad_token=0) -> BeamStep
    reorder_beams(states, beams, out=None) -> states of the chosen beams
"""
from __future__ import annotations

import ctypes
import json
import math
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsgemm_f32.so")

SGEMM_OK = 0
STATUS_NAMES = {0: "SGEMM_OK", -1: "SGEMM_EINVAL_DIM", -2: "SGEMM_EINVAL_LD",
                -3: "SGEMM_EINVAL_PTR", -4: "SGEMM_EALIAS", -5: "SGEMM_ELAUNCH",
                -6: "SGEMM_EINVAL_ARG", -7: "SGEMM_ETOO_LARGE", -8: "SGEMM_ESCRATCH"}

_lib = None


class SgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _load().sgemm_f32_status_string(status).decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({msg})")


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m fp32_gemm_f32_amd.build` "
                               "(or __graft_entry__.build()) first")
        # torch carries its own HIP runtime under the same soname as the system's. Loaded
        # first, it is the one the library binds to; loaded after the library, it would be a
        # second runtime in the process, and the library's own would see no device.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        lib = ctypes.CDLL(LIB_PATH)
        i, p = ctypes.c_int, ctypes.c_void_p
        gemm = [i, i, i, p, i, p, i, p, i]
        lib.sgemm_f32.argtypes = gemm + [p]
        lib.sgemm_f32.restype = i
        lib.sgemm_f32_naive.argtypes = gemm + [p]
        lib.sgemm_f32_naive.restype = i
        lib.sgemm_f32_tiled.argtypes = gemm + [i, i, p]
        lib.sgemm_f32_tiled.restype = i
        lib.sgemm_f32_splitk.argtypes = gemm + [i, p, ctypes.c_size_t, p]
        lib.sgemm_f32_splitk.restype = i
        lib.sgemm_f32_splitk_workspace_size.argtypes = [i, i, i, i]
        lib.sgemm_f32_splitk_workspace_size.restype = ctypes.c_size_t
        lib.sgemm_f32_streamk.argtypes = gemm + [i, p, ctypes.c_size_t, p]
        lib.sgemm_f32_streamk.restype = i
        lib.sgemm_f32_streamk_workspace_size.argtypes = [i, i, i, i, i, i, i]
        lib.sgemm_f32_streamk_workspace_size.restype = ctypes.c_size_t
        lib.sgemm_f32_streamk_noalloc.argtypes = gemm + [i, p]
        lib.sgemm_f32_streamk_noalloc.restype = i
        lib.sgemm_f32_streamk_noalloc_scratch_bytes.argtypes = []
        lib.sgemm_f32_streamk_noalloc_scratch_bytes.restype = ctypes.c_size_t
        lib.sgemm_f32_streamk_describe.argtypes = [i, i, i, i, i, ctypes.c_char_p, i]
        lib.sgemm_f32_streamk_describe.restype = i
        lib.sgemm_f32_regtiled.argtypes = gemm + [i, i, p]
        lib.sgemm_f32_regtiled.restype = i
        lib.sgemm_f32_lds_transpose.argtypes = [i, i, p, i, p, i, i, i, p]
        lib.sgemm_f32_lds_transpose.restype = i
        lib.sgemm_f32_variant.argtypes = [i] + gemm + [p]
        lib.sgemm_f32_variant.restype = i
        lib.sgemm_f32_variant_count.argtypes = []
        lib.sgemm_f32_variant_count.restype = i
        lib.sgemm_f32_variant_name.argtypes = [i]
        lib.sgemm_f32_variant_name.restype = ctypes.c_char_p
        lib.sgemm_f32_variant_info.argtypes = [i, ctypes.c_char_p, i]
        lib.sgemm_f32_variant_info.restype = i
        lib.sgemm_f32_status_string.argtypes = [i]
        lib.sgemm_f32_status_string.restype = ctypes.c_char_p
        lib.sgemm_f32_plan_describe.argtypes = gemm + [i, ctypes.c_char_p, i]
        lib.sgemm_f32_plan_describe.restype = i
        lib.sgemm_f32_variant_describe.argtypes = [i] * 8 + [ctypes.c_char_p, i]
        lib.sgemm_f32_variant_describe.restype = i
        l, z = ctypes.c_int64, ctypes.c_size_t
        lib.gemm_i8_quantize_rows.argtypes = [i, i, p, i, l, p, l, p, p]
        lib.gemm_i8_quantize_rows.restype = i
        lib.gemm_i8.argtypes = [i, i, i, p, l, p, p, l, p, p, p, i, l, p, z, p]
        lib.gemm_i8.restype = i
        lib.gemm_i8_workspace_size.argtypes = [i, i, i, p, l, p, l]
        lib.gemm_i8_workspace_size.restype = z
        lib.gemm_i8_plan_describe.argtypes = [i, i, i, l, l, i, ctypes.c_char_p, i]
        lib.gemm_i8_plan_describe.restype = i
        lib.token_logprobs.argtypes = [i, i, p, i, l, p, i, p, p, p, i, p, p, p, z, p]
        lib.token_logprobs.restype = i
        lib.token_logprobs_workspace_size.argtypes = [i, i, i, i]
        lib.token_logprobs_workspace_size.restype = z
        lib.token_logprobs_backward.argtypes = [i, i, p, i, l, p, i, p, p, p, p, p, p, l, p]
        lib.token_logprobs_backward.restype = i
        lib.token_logprobs_low.argtypes = [i, i, p, i, l, p, i, p, p, p, p, i, p, p, p, z, p]
        lib.token_logprobs_low.restype = i
        lib.token_logprobs_backward_low.argtypes = [i, i, p, i, l, p, i, p, p, p, p, p, p, p, l, p]
        lib.token_logprobs_backward_low.restype = i
        lib.gemm_mx4_quantize.argtypes = [i, i, p, i, l, p, l, p, l, p]
        lib.gemm_mx4_quantize.restype = i
        lib.gemm_mx4_dequantize.argtypes = [i, i, p, l, p, l, p, i, l, p]
        lib.gemm_mx4_dequantize.restype = i
        lib.gemm_mx4.argtypes = [i, i, i, p, l, p, l, p, l, p, l, p, p, i, l, p, z, p]
        lib.gemm_mx4.restype = i
        lib.gemm_mx4_workspace_size.argtypes = [i, i, i, p, l, p, l, p, l, p, l]
        lib.gemm_mx4_workspace_size.restype = z
        lib.gemm_mx4_plan_describe.argtypes = [i, i, i, i, ctypes.c_char_p, i]
        lib.gemm_mx4_plan_describe.restype = i
        lib.beam_step.argtypes = [i, i, i, p, i, l, p, p, l, i, p, p, p, p, z, p]
        lib.beam_step.restype = i
        lib.beam_step_workspace_size.argtypes = [i, i, i, i, i]
        lib.beam_step_workspace_size.restype = z
        lib.reorder_beams.argtypes = [i, i, p, i, p, i, p]
        lib.reorder_beams.restype = i
        lib.sgemm_f32_abi_version.argtypes = []
        lib.sgemm_f32_abi_version.restype = i
        _lib = lib
    return _lib


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _load()


def _check(rc: int, where: str) -> None:
    if rc != SGEMM_OK:
        raise SgemmError(rc, where)


# ------------------------------------------------------------------ raw C-ABI layer -------

def sgemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> None:
    _check(_load().sgemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream or None), "sgemm_f32")


def sgemm_f32_naive(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> None:
    _check(_load().sgemm_f32_naive(M, N, K, A, lda, B, ldb, C, ldc, stream or None),
           "sgemm_f32_naive")


def sgemm_f32_tiled(M, N, K, A, lda, B, ldb, C, ldc, tile=32, pad=0, stream=0) -> None:
    _check(_load().sgemm_f32_tiled(M, N, K, A, lda, B, ldb, C, ldc, tile, pad, stream or None),
           "sgemm_f32_tiled")


def sgemm_f32_splitk(M, N, K, A, lda, B, ldb, C, ldc, splits, workspace, workspace_bytes,
                     stream=0) -> None:
    _check(_load().sgemm_f32_splitk(M, N, K, A, lda, B, ldb, C, ldc, splits, workspace or None,
                                    workspace_bytes, stream or None), "sgemm_f32_splitk")


def sgemm_f32_splitk_workspace_size(M, N, K, splits) -> int:
    return _load().sgemm_f32_splitk_workspace_size(M, N, K, splits)


def sgemm_f32_streamk(M, N, K, A, lda, B, ldb, C, ldc, variant, workspace, workspace_bytes,
                      stream=0) -> None:
    _check(_load().sgemm_f32_streamk(M, N, K, A, lda, B, ldb, C, ldc, variant,
                                     workspace or None, workspace_bytes, stream or None),
           "sgemm_f32_streamk")


def sgemm_f32_streamk_workspace_size(M, N, K, lda=None, ldb=None, ldc=None, variant=-1) -> int:
    lda = K if lda is None else lda
    ldb = N if ldb is None else ldb
    ldc = N if ldc is None else ldc
    return _load().sgemm_f32_streamk_workspace_size(M, N, K, lda, ldb, ldc, variant)


def sgemm_f32_streamk_noalloc(M, N, K, A, lda, B, ldb, C, ldc, variant=-1, stream=0) -> None:
    _check(_load().sgemm_f32_streamk_noalloc(M, N, K, A, lda, B, ldb, C, ldc, variant,
                                             stream or None), "sgemm_f32_streamk_noalloc")


def sgemm_f32_streamk_noalloc_scratch_bytes() -> int:
    return _load().sgemm_f32_streamk_noalloc_scratch_bytes()


def sgemm_f32_streamk_describe(M, N, K, variant=-1, num_cus=0) -> dict:
    buf = ctypes.create_string_buffer(1024)
    rc = _load().sgemm_f32_streamk_describe(M, N, K, variant, num_cus, buf, len(buf))
    if rc < 0:
        raise SgemmError(rc, "sgemm_f32_streamk_describe")
    return json.loads(buf.value.decode())


def sgemm_f32_regtiled(M, N, K, A, lda, B, ldb, C, ldc, tm=4, tn=4, stream=0) -> None:
    _check(_load().sgemm_f32_regtiled(M, N, K, A, lda, B, ldb, C, ldc, tm, tn, stream or None),
           "sgemm_f32_regtiled")


def sgemm_f32_lds_transpose(rows, cols, src, ldi, dst, ldo, tile=32, pad=0, stream=0) -> None:
    _check(_load().sgemm_f32_lds_transpose(rows, cols, src, ldi, dst, ldo, tile, pad,
                                           stream or None), "sgemm_f32_lds_transpose")


def sgemm_f32_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> None:
    _check(_load().sgemm_f32_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream or None),
           "sgemm_f32_variant")


def variant_names() -> list[str]:
    lib = _load()
    return [lib.sgemm_f32_variant_name(i).decode() for i in range(lib.sgemm_f32_variant_count())]


def sgemm_f32_variant_info(variant) -> dict:
    buf = ctypes.create_string_buffer(1024)
    rc = _load().sgemm_f32_variant_info(variant, buf, len(buf))
    if rc < 0:
        raise SgemmError(rc, "sgemm_f32_variant_info")
    return json.loads(buf.value.decode())


def planned_variants() -> list[int]:
    """Indices of the variants the automatic plan may pick."""
    return [i for i in range(len(variant_names())) if sgemm_f32_variant_info(i)["planned"]]


def streamk_variants() -> list[int]:
    """Indices of the variants with a stream-K form (those sgemm_f32_streamk accepts)."""
    return [i for i in range(len(variant_names())) if sgemm_f32_variant_info(i)["streamk"]]


def sgemm_f32_plan_describe(M, N, K, A=0, lda=None, B=0, ldb=None, C=0, ldc=None,
                            num_cus=0) -> dict:
    lda = K if lda is None else lda
    ldb = N if ldb is None else ldb
    ldc = N if ldc is None else ldc
    buf = ctypes.create_string_buffer(1024)
    rc = _load().sgemm_f32_plan_describe(M, N, K, A or None, lda, B or None, ldb, C or None,
                                         ldc, num_cus, buf, len(buf))
    if rc < 0:
        raise SgemmError(rc, "sgemm_f32_plan_describe")
    return json.loads(buf.value.decode())


def sgemm_f32_variant_describe(variant, M, N, K, lda=None, ldb=None, ldc=None,
                               num_cus=0) -> dict:
    lda = K if lda is None else lda
    ldb = N if ldb is None else ldb
    ldc = N if ldc is None else ldc
    buf = ctypes.create_string_buffer(1024)
    rc = _load().sgemm_f32_variant_describe(variant, M, N, K, lda, ldb, ldc, num_cus, buf,
                                            len(buf))
    if rc < 0:
        raise SgemmError(rc, "sgemm_f32_variant_describe")
    return json.loads(buf.value.decode())


def abi_version() -> int:
    return _load().sgemm_f32_abi_version()


def gemm_i8_quantize_rows(M, K, X, x_dtype, ldx, Q, ldq, scales, stream=0) -> None:
    _check(_load().gemm_i8_quantize_rows(M, K, X or None, x_dtype, ldx, Q or None, ldq,
                                         scales or None, stream or None),
           "gemm_i8_quantize_rows")


def gemm_i8(M, N, K, A, lda, a_scales, B, ldb, b_scales, bias, C, c_dtype, ldc, workspace=0,
            workspace_bytes=0, stream=0) -> None:
    _check(_load().gemm_i8(M, N, K, A or None, lda, a_scales or None, B or None, ldb,
                           b_scales or None, bias or None, C or None, c_dtype, ldc,
                           workspace or None, workspace_bytes, stream or None), "gemm_i8")


def gemm_i8_workspace_size(M, N, K, A=0, lda=None, B=0, ldb=None) -> int:
    """For packed operands at aligned addresses unless told otherwise."""
    return _load().gemm_i8_workspace_size(M, N, K, A or None, K if lda is None else lda, B or None,
                                          K if ldb is None else ldb)


def gemm_i8_plan_describe(M, N, K, lda=None, ldb=None, num_cus=0) -> dict:
    buf = ctypes.create_string_buffer(1024)
    _check(_load().gemm_i8_plan_describe(M, N, K, K if lda is None else lda,
                                         K if ldb is None else ldb, num_cus, buf, len(buf)),
           "gemm_i8_plan_describe")
    return json.loads(buf.value.decode())


def token_logprobs_raw(M, V, logits, dtype, ld, tokens, token_bytes, logprobs, entropy, lse, top=0,
                       top_logprobs=0, top_tokens=0, workspace=0, workspace_bytes=0,
                       stream=0, lse_low=0) -> None:
    _check(_load().token_logprobs_low(M, V, logits or None, dtype, ld, tokens or None, token_bytes,
                                      logprobs or None, entropy or None, lse or None,
                                      lse_low or None, top, top_logprobs or None,
                                      top_tokens or None, workspace or None, workspace_bytes,
                                      stream or None), "token_logprobs")


def token_logprobs_workspace_size(M, V, dtype, top) -> int:
    return _load().token_logprobs_workspace_size(M, V, dtype, top)


def token_logprobs_backward_raw(M, V, logits, dtype, ld, tokens, token_bytes, lse, entropy,
                                g_logprob, g_entropy, g_lse, grad, ldg, stream=0,
                                lse_low=0) -> None:
    _check(_load().token_logprobs_backward_low(M, V, logits or None, dtype, ld, tokens or None,
                                               token_bytes, lse or None, lse_low or None,
                                               entropy or None, g_logprob or None,
                                               g_entropy or None, g_lse or None, grad or None,
                                               ldg, stream or None),
           "token_logprobs_backward")


def gemm_mx4_quantize(M, K, X, x_dtype, ldx, Q, ldq, scales, lds, stream=0) -> None:
    _check(_load().gemm_mx4_quantize(M, K, X or None, x_dtype, ldx, Q or None, ldq, scales or None, lds,
                                     stream or None), "gemm_mx4_quantize")


def gemm_mx4_dequantize(M, K, Q, ldq, scales, lds, Y, y_dtype, ldy, stream=0) -> None:
    _check(_load().gemm_mx4_dequantize(M, K, Q or None, ldq, scales or None, lds, Y or None, y_dtype, ldy,
                                       stream or None), "gemm_mx4_dequantize")


def gemm_mx4(M, N, K, A, lda, a_scales, lda_scales, B, ldb, b_scales, ldb_scales, bias, C, c_dtype, ldc,
             workspace=0, workspace_bytes=0, stream=0) -> None:
    _check(_load().gemm_mx4(M, N, K, A or None, lda, a_scales or None, lda_scales, B or None, ldb,
                            b_scales or None, ldb_scales, bias or None, C or None, c_dtype, ldc,
                            workspace or None, workspace_bytes, stream or None), "gemm_mx4")


def gemm_mx4_workspace_size(M, N, K, A=0, lda=None, a_scales=0, lda_scales=None, B=0, ldb=None, b_scales=0,
                            ldb_scales=None) -> int:
    """For packed operands at aligned addresses unless told otherwise."""
    row, blocks = K // 2, (K + 31) // 32
    return _load().gemm_mx4_workspace_size(
        M, N, K, A or None, row if lda is None else lda, a_scales or None,
        blocks if lda_scales is None else lda_scales, B or None, row if ldb is None else ldb,
        b_scales or None, blocks if ldb_scales is None else ldb_scales)


def gemm_mx4_plan_describe(M, N, K, num_cus=0) -> dict:
    buf = ctypes.create_string_buffer(512)
    _check(_load().gemm_mx4_plan_describe(M, N, K, num_cus, buf, len(buf)), "gemm_mx4_plan_describe")
    return json.loads(buf.value.decode())


def beam_step_raw(B, W, V, logits, dtype, ld, scores, finished, pad_token, top, out_scores, out_beams,
                  out_tokens, workspace=0, workspace_bytes=0, stream=0) -> None:
    _check(_load().beam_step(B, W, V, logits or None, dtype, ld, scores or None, finished or None, pad_token,
                             top, out_scores or None, out_beams or None, out_tokens or None,
                             workspace or None, workspace_bytes, stream or None), "beam_step")


def beam_step_workspace_size(B, W, V, dtype, top) -> int:
    return _load().beam_step_workspace_size(B, W, V, dtype, top)


class _BeamState(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p)] + [
        (name, ctypes.c_int64) for name in ("src_row", "dst_row", "count1", "src_step1", "dst_step1", "count2",
                                            "src_step2", "dst_step2", "run")]


def reorder_beams_raw(B, W, beams, beam_bytes, states, stream=0) -> None:
    """states: tuples of beam_state's fields."""
    table = (_BeamState * max(len(states), 1))(*(_BeamState(*s) for s in states))
    _check(_load().reorder_beams(B, W, beams or None, beam_bytes, table, len(states), stream or None),
           "reorder_beams")


# ------------------------------------------------------------------ tensor layer ----------

def _ld(t) -> int:
    """Leading dimension of a row-major 2-D tensor with unit column stride."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("columns must be contiguous (row-major, unit column stride)")
    return max(t.stride(0), t.shape[1], 1)


def matmul(A, B, out=None, kernel: str = "auto", variant: int = -1, tile=32, pad: int = 0):
    """C = A x B for float32 CUDA/HIP tensors, on torch's current stream.

    kernel: "auto" (the hot path, or the given variant), "naive", "tiled", "regtiled"
    (tile = (tm, tn)), "splitk" (variant = number of splits, -1 for automatic) or
    "streamk" (variant = tile variant forced into stream-K, -1 for the automatic choice
    between the plain and the stream-K form). The split-K and stream-K workspaces are
    torch allocations made here.
    """
    import torch

    if A.dtype != torch.float32 or B.dtype != torch.float32:
        raise TypeError("A and B must be float32")
    if not (A.is_cuda and B.is_cuda) or A.device != B.device:
        raise ValueError("A and B must be on the same GPU")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    elif out.shape != (M, N) or out.dtype != torch.float32 or out.device != A.device:
        raise ValueError("out must be a float32 (M, N) tensor on A's device")
    stream = torch.cuda.current_stream(A.device).cuda_stream
    args = (M, N, K, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B), out.data_ptr(), _ld(out))
    with torch.cuda.device(A.device):
        if kernel == "auto":
            if variant < 0:
                sgemm_f32(*args, stream=stream)
            else:
                sgemm_f32_variant(variant, *args, stream=stream)
        elif kernel == "naive":
            sgemm_f32_naive(*args, stream=stream)
        elif kernel == "tiled":
            sgemm_f32_tiled(*args, tile=tile, pad=pad, stream=stream)
        elif kernel == "splitk":
            splits = variant if variant >= 0 else 0
            ws_bytes = sgemm_f32_splitk_workspace_size(M, N, K, splits)
            ws = torch.empty(max(ws_bytes // 4, 1), dtype=torch.float32, device=A.device)
            sgemm_f32_splitk(*args, splits, ws.data_ptr(), ws_bytes, stream=stream)
        elif kernel == "streamk":
            ws_bytes = sgemm_f32_streamk_workspace_size(M, N, K, args[4], args[6], args[8],
                                                        variant)
            ws = torch.empty(max(ws_bytes // 4, 1), dtype=torch.float32, device=A.device)
            sgemm_f32_streamk(*args, variant, ws.data_ptr(), ws_bytes, stream=stream)
        elif kernel == "regtiled":
            tm, tn = tile if isinstance(tile, tuple) else (4, 4)
            sgemm_f32_regtiled(*args, tm=tm, tn=tn, stream=stream)
        else:
            raise ValueError(f"unknown kernel {kernel!r}")
    return out


# ------------------------------------------------------- 8-bit product, token log-probabilities

_calls = None


def _load_calls():
    """The extension module that makes the tensor layer's ordinary calls (csrc/torch_calls.cpp);
    each of its functions returns None where the checks below have to decide."""
    global _calls
    if _calls is None:
        library()
        import torch  # noqa: F401  (the extension links against its libraries)
        try:
            from . import _torch_calls
        except ImportError as e:
            raise RuntimeError("the extension _torch_calls is not built or does not load; run "
                               "`python -m fp32_gemm_f32_amd.build`") from e
        _calls = _torch_calls
    return _calls


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns for M rows: logprobs, entropy and lse are (M,) float32;
    top_logprobs (M, top) float32 and top_tokens (M, top) int64, or None with top = 0."""
    logprobs: object
    entropy: object
    lse: object
    top_logprobs: object = None
    top_tokens: object = None


_dtype_codes = None


def _dtype_code(dtype) -> int:
    """The sgemm_dtype of a torch element type."""
    global _dtype_codes
    if _dtype_codes is None:
        import torch
        _dtype_codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    code = _dtype_codes.get(dtype)
    if code is None:
        raise TypeError(f"expected float32, bfloat16 or float16, got {dtype}")
    return code


def _on_gpu(device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on the same GPU")


def _vector(t, n: int, dtype, name: str):
    """A tensor of n elements of dtype, made contiguous (a broadcast gradient is not)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    return t.resolve_neg().contiguous()


def _rows(t, name: str):
    """A 2-D GPU tensor the kernels can read: rows of unit-stride elements that do not
    overlap, else (a transposed or broadcast tensor) a packed copy."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    rows, cols = t.shape
    if t.is_neg() or (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        return t.resolve_neg().contiguous()
    return t


def _out(t, shape, dtype, device, name: str):
    """A caller's output: exactly this shape and type, written in place."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    if len(shape) == 1:
        if shape[0] > 1 and t.stride(0) != 1:
            raise ValueError(f"{name} must be contiguous")
    elif (shape[1] > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError(f"{name} must have rows of unit-stride elements that do not overlap")
    return t


def _ld_of(t) -> int:
    rows, cols = t.shape
    return max(t.stride(0) if rows > 1 else cols, cols, 1)


class _Device:
    """Makes a tensor's device current for a launch, if it is not already."""
    __slots__ = ("index", "before")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        import torch
        self.before = torch.cuda.current_device()
        if self.before != self.index:
            torch.cuda.set_device(self.index)
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *exc):
        if self.before != self.index:
            import torch
            torch.cuda.set_device(self.before)


def quantize_rows(X, out=None, scales=None):
    """(Q, scales): each row of X (M, K) as 8-bit integers with one float32 scale, so that X
    is about Q * scales[:, None]. X is float32, bfloat16 or float16; a row is a token of
    activations or an output channel of weights. The integers are defined to the bit
    (gemm_i8.h). No gradient flows through it."""
    if out is None and scales is None:
        done = (_calls or _load_calls()).quantize_rows(X)
        if done is not None:
            return done
    import torch

    code = _dtype_code(X.dtype)
    X = _rows(X.detach(), "X")
    M, K = X.shape
    out = (torch.empty((M, K), dtype=torch.int8, device=X.device) if out is None
           else _out(out, (M, K), torch.int8, X.device, "out"))
    scales = (torch.empty((M,), dtype=torch.float32, device=X.device) if scales is None
              else _out(scales, (M,), torch.float32, X.device, "scales"))
    with _Device(X.device) as stream:
        gemm_i8_quantize_rows(M, K, X.data_ptr(), code, _ld_of(X), out.data_ptr(), _ld_of(out),
                              scales.data_ptr(), stream)
    return out, scales


def matmul_i8(A, a_scales, B, b_scales, bias=None, out_dtype=None, out=None):
    """C[i, j] = (sum_k A[i, k] B[j, k]) a_scales[i] b_scales[j] + bias[j], the sum exact in
    32-bit integers. A is (M, K) and B (N, K) int8 (a row of B is an output channel);
    a_scales (M,), b_scales (N,) and bias (N,) float32. C is out_dtype (float32 by default,
    bfloat16 or float16). K is at most 131071. The workspace (for a split K, or for large
    operands off the alignment the kernels load) is a torch allocation made here. No gradient flows through it."""
    import torch

    if out is None:
        done = (_calls or _load_calls()).matmul_i8(A, a_scales, B, b_scales, bias,
                                                   0 if out_dtype is None else _dtype_code(out_dtype))
        if done is not None:
            return done
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    A, B = _rows(A, "A"), _rows(B, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError(f"rows of A and B differ in length: {K} vs {K2}")
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    code = _dtype_code(out_dtype)
    dev = A.device
    _on_gpu(dev, B, a_scales, b_scales, bias)
    a_scales = _vector(a_scales.detach(), M, torch.float32, "a_scales")
    b_scales = _vector(b_scales.detach(), N, torch.float32, "b_scales")
    bias = None if bias is None else _vector(bias.detach(), N, torch.float32, "bias")
    out = (torch.empty((M, N), dtype=out_dtype, device=dev) if out is None
           else _out(out, (M, N), out_dtype, dev, "out"))
    with _Device(dev) as stream:
        ws_bytes = gemm_i8_workspace_size(M, N, K, A.data_ptr(), _ld_of(A), B.data_ptr(), _ld_of(B))
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        gemm_i8(M, N, K, A.data_ptr(), _ld_of(A), a_scales.data_ptr(), B.data_ptr(), _ld_of(B),
                b_scales.data_ptr(), 0 if bias is None else bias.data_ptr(), out.data_ptr(),
                code, _ld_of(out), 0 if ws is None else ws.data_ptr(), ws_bytes, stream)
    return out


def linear_i8(X, B, b_scales, bias=None, out_dtype=None):
    """quantize_rows(X), then its product with the 8-bit weights B (N, K) of scales b_scales:
    a projection of activations X (..., K) in 8 bits. The result has X's type unless
    out_dtype says otherwise. No gradient flows through it."""
    # (the number of rows is given, not left to reshape: with K = 0 it cannot tell)
    q, scales = quantize_rows(X if X.dim() == 2 else X.reshape(math.prod(X.shape[:-1]), X.shape[-1]))
    C = matmul_i8(q, scales, B, b_scales, bias=bias, out_dtype=out_dtype or X.dtype)
    return C if X.dim() == 2 else C.view(*X.shape[:-1], B.shape[0])


def _tokens(tokens, M: int, device):
    import torch

    if tokens.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"tokens must be int64 or int32, got {tokens.dtype}")
    _on_gpu(device, tokens)
    return _vector(tokens, M, tokens.dtype, "tokens"), (8 if tokens.dtype == torch.int64 else 4)


def _logprobs_forward(logits, tokens, top: int, low: bool = False):
    """TokenLogprobs' fields and lse_low, which is None unless asked for."""
    done = (_calls or _load_calls()).token_logprobs(logits, tokens, top, low)
    if done is not None:
        return done
    import torch

    if torch.autograd.forward_ad.unpack_dual(logits).tangent is not None:
        raise NotImplementedError("token_logprobs has no forward-mode derivative: logits must not "
                                  "carry a tangent")
    code = _dtype_code(logits.dtype)
    logits = _rows(logits, "logits")
    M, V = logits.shape
    dev = logits.device
    tokens, token_bytes = _tokens(tokens, M, dev)
    if not 0 <= top <= 64 or (M and top > V):
        raise ValueError(f"top must be between 0 and min(64, {V}), got {top}")
    logprobs, entropy, lse = (torch.empty((M,), dtype=torch.float32, device=dev)
                              for _ in range(3))
    top_logprobs = top_tokens = None
    if top:
        top_logprobs = torch.empty((M, top), dtype=torch.float32, device=dev)
        top_tokens = torch.empty((M, top), dtype=torch.int64, device=dev)
    lse_low = torch.empty((M,), dtype=torch.float32, device=dev) if low else None
    with _Device(dev) as stream:
        ws_bytes = token_logprobs_workspace_size(M, V, code, top)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        token_logprobs_raw(M, V, logits.data_ptr(), code, _ld_of(logits), tokens.data_ptr(),
                           token_bytes, logprobs.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
                           top, top_logprobs.data_ptr() if top else 0,
                           top_tokens.data_ptr() if top else 0,
                           0 if ws is None else ws.data_ptr(), ws_bytes, stream,
                           lse_low.data_ptr() if low else 0)
    return logprobs, entropy, lse, top_logprobs, top_tokens, lse_low


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logprobs, grad_entropy=None,
                            grad_lse=None, out=None, lse_low=None):
    """The gradient with respect to logits of
    sum(grad_logprobs * logprobs + grad_entropy * entropy + grad_lse * lse), from the lse and
    entropy that token_logprobs returned for these logits; a gradient that is None counts as
    zeros (entropy may be None where grad_entropy is). out may be logits itself: the gradient
    then takes its place. No gradient flows through it.

    The probabilities are exp(logits - lse), and off by lse's rounding to FP32: 1e-6 for logits of
    ordinary size, 0.2 % at 60000, and a row of the type's lowest value loses them altogether.
    lse_low (M,) float32 is what that rounding left off: token_logprobs_raw writes it where asked,
    and autograd keeps and passes it."""
    if out is None:
        done = (_calls or _load_calls()).token_logprobs_backward(logits, tokens, lse, entropy,
                                                                 grad_logprobs, grad_entropy,
                                                                 grad_lse, lse_low)
        if done is not None:
            return done
    import torch

    code = _dtype_code(logits.dtype)
    source = logits.detach()
    logits = _rows(source, "logits")
    M, V = logits.shape
    dev = logits.device
    tokens, token_bytes = _tokens(tokens, M, dev)
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    _on_gpu(dev, lse, entropy, grad_logprobs, grad_entropy, grad_lse, lse_low)
    vectors = [None if t is None else _vector(t.detach(), M, torch.float32, name)
               for t, name in ((lse, "lse"), (entropy, "entropy"),
                               (grad_logprobs, "grad_logprobs"),
                               (grad_entropy, "grad_entropy"), (grad_lse, "grad_lse"),
                               (lse_low, "lse_low"))]
    if vectors[0] is None:
        raise ValueError("lse is needed")
    out = (torch.empty((M, V), dtype=logits.dtype, device=dev) if out is None
           else _out(out, (M, V), logits.dtype, dev, "out"))
    with _Device(dev) as stream:
        token_logprobs_backward_raw(M, V, logits.data_ptr(), code, _ld_of(logits),
                                    tokens.data_ptr(), token_bytes,
                                    *(0 if t is None else t.data_ptr() for t in vectors[:5]),
                                    out.data_ptr(), _ld_of(out), stream,
                                    0 if lse_low is None else vectors[5].data_ptr())
    return out


_autograd = None


def _autograd_function():
    """The autograd form of token_logprobs, made on first use (the module imports without
    torch)."""
    global _autograd
    if _autograd is None:
        import torch
        from torch.autograd.function import once_differentiable

        class TokenLogprobsFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, tokens, top):
                *out, lse_low = _logprobs_forward(logits, tokens, top, True)
                ctx.save_for_backward(logits, tokens, out[2], out[1], lse_low)
                ctx.set_materialize_grads(False)
                if top:
                    ctx.mark_non_differentiable(*out[3:])
                return tuple(out)

            @staticmethod
            @once_differentiable
            def backward(ctx, g_logprobs, g_entropy, g_lse, *_):
                if g_logprobs is None and g_entropy is None and g_lse is None:
                    return None, None, None
                logits, tokens, lse, entropy, lse_low = ctx.saved_tensors
                return token_logprobs_backward(logits, tokens, lse, entropy, g_logprobs, g_entropy,
                                               g_lse, lse_low=lse_low), None, None

        _autograd = TokenLogprobsFunction
    return _autograd


def token_logprobs(logits, tokens, top: int = 0) -> TokenLogprobs:
    """Log-probabilities of one token a row under softmax(logits), with each row's entropy
    (nats), log-sum-exp and `top` (at most 64) likeliest alternatives, in one pass over the
    logits. logits is (M, V) float32, bfloat16 or float16; tokens (M,) int64 or int32. A
    token below 0 marks a row without one: logprob 0 and no gradient from it; one of V or
    more gives NaN. Alternatives of equal logits come by ascending index.

    logprobs, entropy and lse carry gradients to logits where it requires them
    (token_logprobs_backward, in one pass too); the alternatives carry none. There is no
    forward-mode derivative (logits with a tangent are refused). In a graph capture
    call token_logprobs_backward itself rather than .backward(): autograd accumulates into a leaf
    on the stream it first saw it on, which a capture must not wait for."""
    import torch

    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_autograd_function().apply(logits, tokens, top))
    return TokenLogprobs(*_logprobs_forward(logits, tokens, top)[:5])


# ------------------------------------------------------- 4-bit product, beam search

def _padded(rows: int, cols: int, device):
    """Rows of bytes whose starts the product's kernels load without a copy: (rows, cols), packed where
    4 divides cols, else 16-byte aligned rows."""
    import torch

    if cols % 4 == 0 or rows < 2:
        return torch.empty((rows, cols), dtype=torch.uint8, device=device)
    return torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=device)[:, :cols]


def _no_tangent(what: str, *tensors) -> None:
    """Refuses tensors that carry a forward-mode tangent, which would be lost."""
    import torch

    for t in tensors:
        if t is not None and torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{what} has no forward-mode derivative: its tensors must not carry a "
                                      "tangent")


def _check_outputs(*outs) -> None:
    """A caller's outputs take no part in a graph of gradients: what it holds for them would be the
    gradient of what was there before."""
    import torch

    for t in outs:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("an out that requires grad cannot be written: no gradient flows through this "
                               "operator")


def _written(*outs) -> None:
    """Tells autograd that a caller's outputs hold other values now, so that a backward pass that saved one
    of them refuses to use it."""
    from torch.autograd.graph import increment_version

    increment_version([t for t in outs if t is not None])


def _int_sizes(*sizes):
    """Sizes that the C ABI takes, which counts rows and columns in 32 bits."""
    for n in sizes:
        if n > 0x7fffffff:
            raise ValueError(f"at most 2147483647 rows and columns, not {n}")
    return sizes


def quantize_mx4(X, out=None, scales=None):
    """(Q, scales): X (M, K) in microscaled 4-bit floating point (E2M1 elements, a power of two for each
    32 of a row). Q is (M, ceil(K / 2)) uint8, element 2 i of a row in the low half of byte i; scales
    (M, ceil(K / 32)) uint8, s for 2^(s - 127). X is float32, bfloat16 or float16; a row is a token of
    activations or an output channel of weights. The codes are defined to the bit (gemm_mx4.h).
    Where 4 does not divide a row's bytes the result is a view of padded rows, which the product reads
    in place. No gradient flows through it; a forward-mode tangent is refused."""
    if out is None and scales is None:
        done = (_calls or _load_calls()).quantize_mx4(X)
        if done is not None:
            return done
    import torch

    _no_tangent("quantize_mx4", X)
    _check_outputs(out, scales)
    code = _dtype_code(X.dtype)
    X = _rows(X.detach(), "X")
    M, K = _int_sizes(*X.shape)
    row, blocks = (K + 1) // 2, (K + 31) // 32
    given = out, scales
    out = _padded(M, row, X.device) if out is None else _out(out, (M, row), torch.uint8, X.device, "out")
    scales = (_padded(M, blocks, X.device) if scales is None
              else _out(scales, (M, blocks), torch.uint8, X.device, "scales"))
    with _Device(X.device) as stream:
        gemm_mx4_quantize(M, K, X.data_ptr(), code, _ld_of(X), out.data_ptr(), _ld_of(out),
                          scales.data_ptr(), _ld_of(scales), stream)
    _written(*given)
    return out, scales


def _packed_rows(q, scales, name: str):
    """A packed matrix and its scales, as the kernels read them."""
    import torch

    if q.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name} and its scales must be uint8, got {q.dtype} and {scales.dtype}")
    q, scales = _rows(q, name), _rows(scales, f"{name}'s scales")
    _on_gpu(q.device, scales)
    if scales.shape[0] != q.shape[0] or scales.shape[1] != (q.shape[1] + 15) // 16:
        raise ValueError(f"{name}'s scales must have shape ({q.shape[0]}, {(q.shape[1] + 15) // 16}), "
                         f"got {tuple(scales.shape)}")
    return q, scales


def dequantize_mx4(Q, scales, dtype=None, columns=None, out=None):
    """The values that Q (M, R) uint8 with its scales stands for: (M, columns) of dtype (float32 by
    default, bfloat16 or float16), columns 2 R unless it is given as 2 R - 1. No gradient flows
    through it; a forward-mode tangent is refused."""
    import torch

    if out is None:
        done = (_calls or _load_calls()).dequantize_mx4(Q, scales, 0 if dtype is None else _dtype_code(dtype),
                                                        columns)
        if done is not None:
            return done
    given = out
    _no_tangent("dequantize_mx4", out)
    _check_outputs(given)
    Q, scales = _packed_rows(Q, scales, "Q")
    M, R = Q.shape
    if columns is None:
        columns = 2 * R
    if (columns + 1) // 2 != R or columns < 0:
        raise ValueError(f"rows of {R} bytes hold {2 * R} or {2 * R - 1} columns, not {columns}")
    _int_sizes(M, columns)
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    code = _dtype_code(dtype)
    out = (torch.empty((M, columns), dtype=dtype, device=Q.device) if out is None
           else _out(out, (M, columns), dtype, Q.device, "out"))
    with _Device(Q.device) as stream:
        gemm_mx4_dequantize(M, columns, Q.data_ptr(), _ld_of(Q), scales.data_ptr(), _ld_of(scales),
                            out.data_ptr(), code, _ld_of(out), stream)
    _written(given)
    return out


def matmul_mx4(A, a_scales, B, b_scales, bias=None, out_dtype=None, out=None):
    """C[i, j] = sum_k A[i, k] B[j, k] + bias[j] of the values that quantize_mx4's operands stand for, on
    the matrix cores in 4 bits, summed in FP32. A is (M, R) and B (N, R) uint8 of 2 R elements a row (a
    row of B is an output channel), their scales (M or N, ceil(R / 16)) uint8, bias (N,) float32. C is
    out_dtype (float32 by default, bfloat16 or float16). The workspace (for a split K, or for
    operands off a word's boundary) is a torch allocation made here. No gradient flows through
    it; a forward-mode tangent is refused."""
    import torch

    if out is None:
        done = (_calls or _load_calls()).matmul_mx4(A, a_scales, B, b_scales, bias,
                                                    0 if out_dtype is None else _dtype_code(out_dtype))
        if done is not None:
            return done
    given = out
    _no_tangent("matmul_mx4", bias, out)
    _check_outputs(given)
    A, a_scales = _packed_rows(A, a_scales, "A")
    B, b_scales = _packed_rows(B, b_scales, "B")
    M, R = A.shape
    N, R2 = B.shape
    if R != R2:
        raise ValueError(f"rows of A and B differ in length: {R} vs {R2} bytes")
    _int_sizes(M, N, 2 * R)
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    code = _dtype_code(out_dtype)
    dev = A.device
    _on_gpu(dev, B, bias)
    bias = None if bias is None else _vector(bias.detach(), N, torch.float32, "bias")
    out = (torch.empty((M, N), dtype=out_dtype, device=dev) if out is None
           else _out(out, (M, N), out_dtype, dev, "out"))
    operands = (A.data_ptr(), _ld_of(A), a_scales.data_ptr(), _ld_of(a_scales),
                B.data_ptr(), _ld_of(B), b_scales.data_ptr(), _ld_of(b_scales))
    with _Device(dev) as stream:
        ws_bytes = gemm_mx4_workspace_size(M, N, 2 * R, *operands)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        gemm_mx4(M, N, 2 * R, *operands, 0 if bias is None else bias.data_ptr(), out.data_ptr(), code,
                 _ld_of(out), 0 if ws is None else ws.data_ptr(), ws_bytes, stream)
    _written(given)
    return out


def linear_mx4(X, B, b_scales, bias=None, out_dtype=None):
    """quantize_mx4(X), then its product with the 4-bit weights B (N, ceil(K / 2)) of scales b_scales: a
    projection of activations X (..., K). The result has X's type unless out_dtype says
    otherwise. No gradient flows through it; a forward-mode tangent is refused."""
    if X.dim() == 2:
        done = (_calls or _load_calls()).linear_mx4(X, B, b_scales, bias,
                                                    -1 if out_dtype is None else _dtype_code(out_dtype))
        if done is not None:
            return done
    # (the number of rows is given, not left to reshape: with K = 0 it cannot tell)
    q, scales = quantize_mx4(X if X.dim() == 2 else X.reshape(math.prod(X.shape[:-1]), X.shape[-1]))
    C = matmul_mx4(q, scales, B, b_scales, bias=bias, out_dtype=out_dtype or X.dtype)
    return C if X.dim() == 2 else C.view(*X.shape[:-1], B.shape[0])


class BeamStep(NamedTuple):
    """What beam_step returns for B requests: scores (B, top) float32, beams and tokens (B, top) int64,
    in descending order of the scores; score -infinity, beam -1 and token -1 where there is none."""
    scores: object
    beams: object
    tokens: object


def beam_step(logits, scores, top=None, finished=None, pad_token: int = 0) -> BeamStep:
    """One step of a beam search: the `top` best continuations (beam, token) of each request by
    scores[b, w] + log softmax(logits[b W + w])[token], in one pass over the logits. logits is (B W, V)
    float32, bfloat16 or float16, a row for each beam; scores (B, W) float32, the logarithms of the
    beams' probabilities so far. top is W unless given; W and top are at most 64.

    finished (B, W) bool marks beams that have ended: such a beam offers itself alone, with its score
    and pad_token. Continuations of probability 0 (logits or scores of -infinity) and of rows that
    hold a NaN or +infinity do not count. Of equal totals the lower beam comes first, of a beam's equal
    logits the lower token. No gradient flows through it; a forward-mode tangent is refused."""
    done = (_calls or _load_calls()).beam_step(logits, scores, top, finished, pad_token)
    if done is not None:
        return BeamStep(*done)
    import torch

    _no_tangent("beam_step", logits, scores)
    if not -2 ** 63 <= pad_token < 2 ** 63:
        raise ValueError(f"pad_token must fit 64 bits, got {pad_token}")
    code = _dtype_code(logits.dtype)
    if scores.dim() != 2:
        raise ValueError(f"scores must be 2-D, got {scores.dim()}-D")
    B, W = scores.shape
    logits = _rows(logits.detach(), "logits")
    dev = logits.device
    if logits.shape[0] != B * W:
        raise ValueError(f"logits must have {B * W} rows, one for each beam, got {logits.shape[0]}")
    V = logits.shape[1]
    _int_sizes(B, V)
    top = W if top is None else top
    if scores.dtype != torch.float32:
        raise TypeError(f"scores must be float32, got {scores.dtype}")
    if finished is not None and finished.dtype != torch.bool:
        raise TypeError(f"finished must be bool, got {finished.dtype}")
    if finished is not None and tuple(finished.shape) != (B, W):
        raise ValueError(f"finished must have shape ({B}, {W}), got {tuple(finished.shape)}")
    if not 1 <= W <= 64 or not 1 <= top <= 64:
        raise ValueError(f"a request has 1 to 64 beams and as many continuations, got {W} and {top}")
    _on_gpu(dev, scores, finished)
    scores = scores.detach().resolve_neg().contiguous()
    finished = None if finished is None else finished.contiguous()
    out = BeamStep(torch.empty((B, top), dtype=torch.float32, device=dev),
                   torch.empty((B, top), dtype=torch.int64, device=dev),
                   torch.empty((B, top), dtype=torch.int64, device=dev))
    with _Device(dev) as stream:
        ws_bytes = beam_step_workspace_size(B, W, V, code, top)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
        beam_step_raw(B, W, V, logits.data_ptr(), code, _ld_of(logits), scores.data_ptr(),
                      0 if finished is None else finished.data_ptr(), pad_token, top,
                      *(t.data_ptr() for t in out), 0 if ws is None else ws.data_ptr(), ws_bytes, stream)
    return out


def _beam_state(src, dst):
    """beam_state's fields for two tensors of one shape, None where they have more than two dimensions
    of pieces."""
    size = src.element_size()
    dims = []                                        # [count, src step, dst step], outermost first
    for n, a, b in zip(src.shape[1:], src.stride()[1:], dst.stride()[1:]):
        if n == 1:
            continue
        if dims and dims[-1][1] == n * a * size and dims[-1][2] == n * b * size:
            dims[-1] = [dims[-1][0] * n, a * size, b * size]
        else:
            dims.append([n, a * size, b * size])
    run = size
    if dims and dims[-1][1:] == [size, size]:
        run *= dims.pop()[0]
    if len(dims) > 2:
        return None
    dims = [[1, 0, 0]] * (2 - len(dims)) + dims
    return (src.data_ptr(), dst.data_ptr(), src.stride(0) * size if src.shape[0] > 1 else 0,
            dst.stride(0) * size if src.shape[0] > 1 else 0, *dims[0], *dims[1], run)


def reorder_beams(states, beams, out=None):
    """The states of the beams that a step chose: row b W + w of each result is row b W + beams[b, w] of
    its state. states is a tensor or a sequence of tensors of any type whose first dimension is B W (key
    and value caches, also views of their first positions; tokens so far), beams (B, W) int64 or
    int32; an index outside 0 to W - 1 stands for w itself. All are moved in one launch.

    Results are new tensors (small ones, 64 MiB in all, may share an allocation), or written to out:
    tensors of the same shapes and types, for which out=states reorders in place and leaves rows that
    stay alone. An out must not overlap itself or another state, nor require grad (but under
    torch.no_grad); a backward pass that saved its values notices the change. No gradient flows
    through it; a forward-mode tangent is refused."""
    done = (_calls or _load_calls()).reorder_beams(states, beams, out)
    if done is not None:
        return done
    import torch

    single = isinstance(states, torch.Tensor)
    sources = [states] if single else list(states)
    targets = None if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    _no_tangent("reorder_beams", *sources, *(targets or ()))
    _check_outputs(*(targets or ()))
    if beams.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"beams must be int64 or int32, got {beams.dtype}")
    if beams.dim() != 2:
        raise ValueError(f"beams must be 2-D, got {beams.dim()}-D")
    if not beams.is_cuda:
        raise ValueError("beams must be on a GPU")
    B, W = beams.shape
    if W > 64:
        raise ValueError(f"a request has at most 64 beams, got {W}")
    _int_sizes(B)
    dev = beams.device
    _on_gpu(dev, *sources)
    beams = beams.resolve_neg().contiguous()
    for t in sources:
        if t.dim() < 1 or t.shape[0] != B * W:
            raise ValueError(f"a state's first dimension must be {B * W}, got shape {tuple(t.shape)}")
    if targets is None:
        sources = [t.detach().resolve_conj().resolve_neg() for t in sources]
        targets = [torch.empty(t.shape, dtype=t.dtype, device=dev) for t in sources]
        whole = [_beam_state(s, t) for s, t in zip(sources, targets)]
        sources = [s if w is not None else s.contiguous() for s, w in zip(sources, whole)]
    else:
        if len(targets) != len(sources):
            raise ValueError(f"{len(sources)} states, but {len(targets)} in out")
        _on_gpu(dev, *targets)
        for s, t in zip(sources, targets):
            if s.shape != t.shape or s.dtype != t.dtype:
                raise ValueError(f"out must match its state: {tuple(s.shape)} {s.dtype}, got "
                                 f"{tuple(t.shape)} {t.dtype}")
            if s.is_neg() != t.is_neg() or s.is_conj() != t.is_conj():
                raise ValueError("out must match its state: one is a negated or conjugated view")
    table = []
    for s, t in zip(sources, targets):
        if s.numel():
            fields = _beam_state(s, t)
            if fields is None:
                raise ValueError(f"a state of strides {s.stride()} has more than two dimensions of pieces: make "
                                 "it contiguous")
            table.append(fields)
    with _Device(dev) as stream:
        reorder_beams_raw(B, W, beams.data_ptr(), beams.element_size(), table, stream)
    if out is not None:
        _written(*targets)
    return targets[0] if single else targets
