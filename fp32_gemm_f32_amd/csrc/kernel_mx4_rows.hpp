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
//  * The next turn is loaded before this one is multiplied.
constexpr int kMx4Turn = 256;
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_rows(Mx4Args p)
{
    static_assert(256 <= 64 * WAVES, "an element of C to a thread");
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
    const uint8_t *A = p.A + ar * p.lda, *SA = p.sa + ar * p.ldsa;
    const uint8_t *B = p.B + br * p.ldb, *SB = p.sb + br * p.ldsb;
    const int blocks = (p.KB + 15) / 16;
    const int em = m0 + tid / 16, en = n0 + tid % 16;
    const bool stores = tid < 256 && em < p.M && en < p.N;
    const float bias = stores && p.bias ? p.bias[en] : 0.0f;

    struct Turn {
        i32x4 a[4], b[4], sa, sb;
    };
    auto load = [&](Turn &x, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) x.b[t] = mx4_load16(B + k + 64 * t + 16 * q);
        x.sb = mx4_load16(SB + k / 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) x.a[t] = mx4_load16(A + k + 64 * t + 16 * q);
        x.sa = mx4_load16(SA + k / 16);
    };
    f32x4 acc = f32x4(0.0f);
    auto multiply = [&](const Turn &x) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const i32x8 a = __builtin_shufflevector(x.a[t], x.a[t], 0, 1, 2, 3, -1, -1, -1, -1);
            const i32x8 b = __builtin_shufflevector(x.b[t], x.b[t], 0, 1, 2, 3, -1, -1, -1, -1);
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, 0, int(uint32_t(x.sa[t]) >> 8 * q), 0,
                                                                   int(uint32_t(x.sb[t]) >> 8 * q));
        }
    };
    constexpr int STRIDE = WAVES * kMx4Turn;
    const int whole = k0 + (k1 - k0) / kMx4Turn * kMx4Turn;        // end of the whole turns
    const int first = k0 + wave * kMx4Turn;
    if (first < whole) {
        Turn x;
        load(x, first);
        for (int k = first + STRIDE; k < whole; k += STRIDE) {
            Turn y;
            load(y, k);
            __builtin_amdgcn_sched_barrier(0);
            multiply(x);
            x = y;
        }
        multiply(x);
    }
    if (whole < k1 && (whole - k0) / kMx4Turn % WAVES == wave) {   // what is left, less than a turn
        Turn x;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = whole + 64 * t + 16 * q;
            x.a[t] = mx4_load_tail(A, k, k1);
            x.b[t] = mx4_load_tail(B, k, k1);
        }
        x.sa = mx4_load_tail(SA, whole / 16, blocks);
        x.sb = mx4_load_tail(SB, whole / 16, blocks);
        multiply(x);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][(4 * q + v) * 16 + r] = acc[v];
    __syncthreads();
    if (!stores) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += sums[w][tid];
    if (p.splits > 1) {
        p.partial[(int64_t(split) * p.M + em) * p.N + en] = sum;
        return;
    }
    mx4_store_one(p.c_dtype, p.C, em * p.ldc + en, sum + bias);
}

// The same for more columns than workgroups that run at once: a workgroup goes on to other columns, with
// A in registers. K is at most a turn to a wave; the next columns are loaded before these are
// multiplied. 16 x 50001 x 4096 to bf16 23.5 us with 8 waves and two workgroups to a compute unit (4.6
// TB/s of B; with A loaded again for each 16 columns 33.3), 16 x 50001 x 8192 45.5 with 16 waves and one
// (61.6; two turns to a wave 47.1, their registers leave too few loads in flight).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_rows_on(Mx4Args p)
{
    constexpr int NT = 64 * WAVES;
    static_assert(256 <= NT, "an element of C to a thread");
    __shared__ float sums[2][WAVES][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int64_t ar = min(r, p.M - 1);
    const uint8_t *const A = p.A + ar * p.lda, *const SA = p.sa + ar * p.ldsa;
    const int blocks = (p.KB + 15) / 16;
    struct Turn {
        i32x4 v[4], s;
    };
    // this wave's turn of a row and its scales: whole, in part, or none of K's
    const int k = wave * kMx4Turn;
    auto load = [&](Turn &x, const uint8_t *row, const uint8_t *scales) __attribute__((always_inline)) {
        if (k + kMx4Turn <= p.KB) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x.v[i] = mx4_load16(row + k + 64 * i + 16 * q);
            x.s = mx4_load16(scales + k / 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x.v[i] = mx4_load_tail(row, k + 64 * i + 16 * q, p.KB);
            x.s = mx4_load_tail(scales, k / 16, blocks);
        }
    };
    auto load_columns = [&](Turn &x, int tile) __attribute__((always_inline)) {
        const int64_t br = min(tile * 16 + r, p.N - 1);
        load(x, p.B + br * p.ldb, p.sb + br * p.ldsb);
    };
    Turn a, b;
    load_columns(b, blockIdx.x);
    load(a, A, SA);
    int buffer = 0;
    for (int tile = blockIdx.x; tile < p.tiles_n; tile += gridDim.x, buffer ^= 1) {
        Turn next;
        load_columns(next, min(tile + int(gridDim.x), p.tiles_n - 1));
        const int em = tid / 16, en = tile * 16 + tid % 16;
        const bool stores = tid < 256 && em < p.M && en < p.N;
        const float bias = stores && p.bias ? p.bias[en] : 0.0f;
        __builtin_amdgcn_sched_barrier(0);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                __builtin_shufflevector(a.v[i], a.v[i], 0, 1, 2, 3, -1, -1, -1, -1),
                __builtin_shufflevector(b.v[i], b.v[i], 0, 1, 2, 3, -1, -1, -1, -1), acc, 4, 4, 0,
                int(uint32_t(a.s[i]) >> 8 * q), 0, int(uint32_t(b.s[i]) >> 8 * q));
#pragma unroll
        for (int v = 0; v < 4; ++v) sums[buffer][wave][(4 * q + v) * 16 + r] = acc[v];
        __syncthreads();       // (the other buffer is read before the next one, and written after it)
        if (stores) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum += sums[buffer][w][tid];
            mx4_store_one(p.c_dtype, p.C, em * p.ldc + en, sum + bias);
        }
        b = next;
    }
}

}  // namespace sgemm
