// kernel_mx4_rows.hpp -- the product of microscaled 4-bit operands (gemm_mx4.h) for few rows of A (a
// decode batch): a kernel that streams B from memory straight into matrix operands.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernel_mx4.hpp"

namespace sgemm {

// A workgroup of WAVES waves computes 16 x 16 of C on v_mfma_scale_f32_16x16x128_f8f6f4; the waves
// take turns of 256 bytes of K (512 elements, 16 scales to a row) and their sums are added in LDS, in
// the waves' order.
//  * MFMA operands: lane l supplies row l % 16 and a block of 32 values with its scale, block l / 16
//    of a step of four, on both sides; accumulator register v of lane l is row 4 (l / 16) + v and
//    column l % 16.
//  * A load instruction reads 64 bytes of each of 16 rows. A lane loads its row's 16 scales of a turn
//    and moves byte l / 16 of each word to the bottom, where the MFMA takes it.
//  * Rows of any address and length: loads serve any alignment, what lies past K is zero (elements of
//    both sides, and scales, lest one that is no number meets a zero).
//  * Rows past M and columns past N repeat the last one; their sums are not stored.
constexpr int kMx4Turn = 256;
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_rows(Mx4Args p)
{
    __shared__ float sums[WAVES][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = p.tiles_m * p.tiles_n;
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int m0 = tm * 16, n0 = tn * 16;
    const int k0 = split * p.chunk, k1 = min(p.KB, k0 + p.chunk);
    const int r = lane & 15, q = lane >> 4;
    const int64_t ar = min(m0 + r, p.M - 1), br = min(n0 + r, p.N - 1);
    const uint8_t *A = p.A + ar * p.lda, *B = p.B + br * p.ldb;
    const uint8_t *SA = p.sa + ar * p.ldsa, *SB = p.sb + br * p.ldsb;
    const int blocks = (p.KB + 15) / 16;

    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = k0 + wave * kMx4Turn; k < k1; k += WAVES * kMx4Turn) {
        i32x4 a[4], b[4], sa, sb;
        if (k + kMx4Turn <= k1) {
#pragma unroll
            for (int t = 0; t < 4; ++t) b[t] = mx4_load16(B + k + 64 * t + 16 * q);
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = mx4_load16(A + k + 64 * t + 16 * q);
            sa = mx4_load16(SA + k / 16);
            sb = mx4_load16(SB + k / 16);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                b[t] = mx4_load_tail(B, k + 64 * t + 16 * q, k1);
                a[t] = mx4_load_tail(A, k + 64 * t + 16 * q, k1);
            }
            sa = mx4_load_tail(SA, k / 16, blocks);
            sb = mx4_load_tail(SB, k / 16, blocks);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const i32x8 ax = {a[t][0], a[t][1], a[t][2], a[t][3], 0, 0, 0, 0};
            const i32x8 bx = {b[t][0], b[t][1], b[t][2], b[t][3], 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ax, bx, acc, 4, 4, 0, int(uint32_t(sa[t]) >> 8 * q), 0,
                                                                   int(uint32_t(sb[t]) >> 8 * q));
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][(4 * q + v) * 16 + r] = acc[v];
    __syncthreads();
    const int em = m0 + tid / 16, en = n0 + tid % 16;
    if (tid >= 256 || em >= p.M || en >= p.N) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += sums[w][tid];
    if (p.splits > 1) {
        p.partial[(int64_t(split) * p.M + em) * p.N + en] = sum;
        return;
    }
    mx4_store_one(p.c_dtype, p.C, em * p.ldc + en, p.bias ? sum + p.bias[en] : sum);
}

}  // namespace sgemm
