/*
 * gemm_i8.h -- C ABI of the MI355X (gfx950) product of 8-bit integers with one scale for
 * each row of A (token) and each row of B (output channel), and of the quantiser that
 * makes such operands.
 *
 * Conventions are sgemm_f32.h's: device pointers owned by the caller, leading dimensions
 * in elements, every argument validated before any HIP call, a negative sgemm_status on
 * refusal, asynchronous launches on `stream` (a hipStream_t; NULL is the default stream),
 * no mutable state between calls, no allocation. Any leading dimension and any address
 * aligned to the element works; rows at 4-byte aligned addresses, of a length that 16 divides,
 * are the fast case.
 *
 * Validation (checked in this order):
 *   dimensions >= 0                                     else SGEMM_EINVAL_DIM
 *   a leading dimension >= max(1, its row's length)     else SGEMM_EINVAL_LD
 *   a type of sgemm_dtype                               else SGEMM_EINVAL_ARG
 *   a pointer whose region is non-empty is non-NULL and aligned to its element
 *                                                       else SGEMM_EINVAL_PTR
 *   an output overlaps no input, no other output and no workspace
 *                                                       else SGEMM_EALIAS
 *   sizes within the limits stated below                else SGEMM_ETOO_LARGE
 */
#ifndef GEMM_I8_H
#define GEMM_I8_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm_dtype.h"
#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises each row of X (M x K, leading dimension ldx, type x_dtype) to 8-bit integers
 * with one scale, all in FP32:
 *     peak_i = max_k |x_ik|,   scale_i = peak_i / 127,
 *     q_ik   = clamp(rint(x_ik * (127 / peak_i)), -127, 127)      (ties to even)
 * so that x_ik is about q_ik * scale_i. Both divisions and the product are rounded once,
 * so the integers are the same on any IEEE machine. Q is M x K with leading dimension ldq,
 * scales holds M floats.
 *
 * A row of zeros, or of numbers so small that 127 / peak_i overflows (below 3.8e-37), gets
 * scale 0 and zeros. A row that holds a NaN gets scale NaN, one that holds an infinity and
 * no NaN scale infinity, both with zeros, so a product with it is NaN throughout. K == 0
 * gives scales of 0.
 *
 * Weights (a row for each output channel) and activations (a row for each token) are both
 * quantised this way. M at most 2^31 - 1 rows, 2^31 - 1 elements to a row.
 */
int gemm_i8_quantize_rows(int M, int K,
                          const void *X, int x_dtype, int64_t ldx,
                          int8_t *Q, int64_t ldq,
                          float *scales,
                          void *stream);

/*
 * C[i*ldc + j] = (sum_{k<K} A[i*lda + k] * B[j*ldb + k]) * (a_scales[i] * b_scales[j]) + bias[j]
 * for 0 <= i < M, 0 <= j < N. A is M x K and B is N x K, both row-major (a row of B is one
 * output channel's weights); any values of int8, -128 too. The sum is exact in 32-bit
 * integers and rounded once to FP32, the product of the scales is rounded once, and the two
 * are multiplied and offset with one rounding (a fused multiply-add; zeros without a bias),
 * then rounded once to C's type c_dtype. bias is NULL or N floats. The result does not depend
 * on the plan: any tiling and split gives the same bits.
 *
 * Limits: K <= 131071 (so that K * 128 * 128 stays below 2^31), 256 rows of A or B below 2^31
 * bytes (lda, ldb < 8388608), fewer than 2^30 blocks of 16 x 16 in C, else SGEMM_ETOO_LARGE.
 *
 * workspace: products with few tiles split K over workgroups and join the partial sums
 * there (32-bit integers) with a second kernel; large products of rows off a word's boundary
 * (or of a K that 16 does not divide) copy them there first, in whole 16-byte chunks.
 * Caller-owned device memory of gemm_i8_workspace_size bytes, 16-byte aligned;
 * SGEMM_EINVAL_ARG if smaller, and it must not overlap A, B, C, the scales or bias. NULL
 * with 0 bytes runs without either, which is right for every shape and slower for those. No
 * initialisation needed, contents unspecified on return; calls that share one must not
 * overlap in time.
 *
 * M == 0 or N == 0 launches nothing; K == 0 writes the bias (or zeros; scales are not read
 * then).
 */
int gemm_i8(int M, int N, int K,
            const int8_t *A, int64_t lda, const float *a_scales,
            const int8_t *B, int64_t ldb, const float *b_scales,
            const float *bias,
            void *C, int c_dtype, int64_t ldc,
            void *workspace, size_t workspace_bytes,
            void *stream);

/* Bytes of workspace gemm_i8 uses for these operands on the current device (0: none, also for
 * arguments it would refuse and where no device answers). Of A and B only the addresses
 * count; nothing is read. */
size_t gemm_i8_workspace_size(int M, int N, int K, const int8_t *A, int64_t lda,
                              const int8_t *B, int64_t ldb);

/*
 * Writes a one-line JSON description of the plan gemm_i8 runs, given its workspace, for
 * operands of this shape at 4-byte aligned addresses into buf: tile, form, copies, splits,
 * workspace bytes, the cost the choice was made by (in microseconds of a card at full clock,
 * which large products do not hold: an order, not a time). num_cus > 0 plans for that many compute
 * units (no GPU needed), otherwise the current device's. Returns SGEMM_OK or a negative
 * status (SGEMM_EINVAL_ARG: the buffer is too small).
 */
int gemm_i8_plan_describe(int M, int N, int K, int64_t lda, int64_t ldb, int num_cus, char *buf,
                          int buflen);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_I8_H */
