/*
 * gemm_mx4.h -- C ABI of the MI355X (gfx950) product of matrices in microscaled 4-bit floating
 * point, and of the quantiser that makes such operands and its inverse.
 *
 * The format: an element is a sign, two bits of exponent and one of mantissa (codes 0 to 7 are 0,
 * 0.5, 1, 1.5, 2, 3, 4, 6; code 8 + c is -c), two to a byte, element 2 i of a row in the low half
 * of its byte i. 32 consecutive elements of a row share a power of two: the scale's byte s stands
 * for 2^(s - 127), 255 for NaN. A row of K elements takes (K + 1) / 2 bytes and (K + 31) / 32
 * scales; where K is odd the last byte's high half is 0.
 *
 * Conventions and the order of validation are gemm_i8.h's; leading dimensions of packed rows and of
 * scales are in bytes. Any leading dimension and any address works. Rows of whole 4-byte words
 * (addresses and leading dimensions that 4 divides, of elements and scales) are the fast case.
 */
#ifndef GEMM_MX4_H
#define GEMM_MX4_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm_dtype.h"
#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises each block of 32 elements of each row of X (M x K, leading dimension ldx, type
 * x_dtype; a row's last block may be shorter):
 *     s = max(floor(log2 max |x|) - 2 + 127, 0),
 *     q_k = the nearest of the format's values to x_k / 2^(s - 127), ties to the even code,
 *           magnitudes above 6 to 6
 * The division is exact, so the codes are the same on any machine. A block of zeros gets s = 0 and
 * zeros (a zero keeps its sign); a block that holds a NaN or an infinity gets s = 255 and zeros, so a
 * product with its row is NaN throughout. Q is M rows of (K + 1) / 2 bytes, ldq apart, scales M rows
 * of (K + 31) / 32, lds apart; bytes between rows are left as they are.
 */
int gemm_mx4_quantize(int M, int K,
                      const void *X, int x_dtype, int64_t ldx,
                      uint8_t *Q, int64_t ldq,
                      uint8_t *scales, int64_t lds,
                      void *stream);

/*
 * The values that K elements of each of M rows stand for, q_k 2^(s - 127), rounded once to Y's type
 * (exact in FP32 and BF16 but for scales above 2^125, which may give infinities).
 */
int gemm_mx4_dequantize(int M, int K,
                        const uint8_t *Q, int64_t ldq,
                        const uint8_t *scales, int64_t lds,
                        void *Y, int y_dtype, int64_t ldy,
                        void *stream);

/*
 * C[i*ldc + j] = sum over blocks b of 2^(a_scales[i,b] + b_scales[j,b] - 254)
 *                sum over the block's k of a_ik b_jk            + bias[j]
 * for 0 <= i < M, 0 <= j < N. A is M x K and B is N x K (a row of B is one output channel's
 * weights), K even (else SGEMM_EINVAL_DIM). The products are exact; they are summed in FP32, the
 * bias is added with one rounding and the result rounded once to C's type c_dtype. bias is NULL or
 * N floats. Repeated calls with the same arguments give the same bits; another plan (other shapes
 * or alignments) may sum in another order.
 *
 * Limits: M and N below 2^27, leading dimensions of A, B and their scales below 8388608, fewer than
 * 2^30 blocks of 16 x 16 in C, and a C that one launch's workgroups cover (any of up to 2^35
 * elements), else SGEMM_ETOO_LARGE.
 *
 * workspace: products with few tiles split K over workgroups and join the partial sums there with a
 * second kernel; operands off a word's boundary are copied there first, and so are a large product's
 * scales, in another order. Caller-owned device memory
 * of gemm_mx4_workspace_size bytes, 16-byte aligned, SGEMM_EINVAL_ARG if smaller (where that is 0,
 * NULL with 0 bytes). It must not overlap the operands or C. No initialisation needed, contents
 * unspecified on return; calls that share one must not overlap in time.
 *
 * M == 0 or N == 0 launches nothing; K == 0 writes the bias (or zeros).
 */
int gemm_mx4(int M, int N, int K,
             const uint8_t *A, int64_t lda, const uint8_t *a_scales, int64_t lda_scales,
             const uint8_t *B, int64_t ldb, const uint8_t *b_scales, int64_t ldb_scales,
             const float *bias,
             void *C, int c_dtype, int64_t ldc,
             void *workspace, size_t workspace_bytes,
             void *stream);

/* Bytes of workspace gemm_mx4 needs for these operands on the current device (0: none, also for
 * arguments it would refuse and where no device answers). Of the operands only the addresses
 * count; nothing is read. */
size_t gemm_mx4_workspace_size(int M, int N, int K,
                               const uint8_t *A, int64_t lda, const uint8_t *a_scales, int64_t lda_scales,
                               const uint8_t *B, int64_t ldb, const uint8_t *b_scales, int64_t ldb_scales);

/*
 * Writes a one-line JSON description of the plan gemm_mx4 runs for packed operands of this shape at
 * 4-byte aligned addresses whose rows are whole words into buf: tile, splits, workspace bytes, the
 * cost the choice was made by (an order, not a time). num_cus > 0 plans for that many compute units
 * (no GPU needed), otherwise the current device's. Returns SGEMM_OK or a negative status
 * (SGEMM_EINVAL_ARG: the buffer is too small).
 */
int gemm_mx4_plan_describe(int M, int N, int K, int num_cus, char *buf, int buflen);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MX4_H */
