/*
 * sgemm_dtype.h -- element types of the entry points that take more than FP32
 * (gemm_i8.h, token_logprobs.h). Statuses are sgemm_f32.h's sgemm_status.
 */
#ifndef SGEMM_DTYPE_H
#define SGEMM_DTYPE_H

typedef enum {
    SGEMM_DTYPE_F32 = 0,
    SGEMM_DTYPE_BF16 = 1,
    SGEMM_DTYPE_F16 = 2
} sgemm_dtype;

#endif /* SGEMM_DTYPE_H */
