// kernel_i8_rows.hpp -- the 8-bit product (gemm_i8.h) for few rows of A (a decode batch): a
// kernel that streams B from memory straight into matrix operands.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kernel_i8.hpp"

namespace sgemm {

// A workgroup of WAVES waves computes 16 RB rows x 16 CB columns of C on
// v_mfma_i32_16x16x64_i8; the waves share K, panel by panel of 64 U bytes in turn, and add
// their sums in LDS (integers: the order does not matter).
//  * MFMA operands: lane l supplies row l % 16 and the 16 values of k from 16 (l / 16) of a
//    step of 64, on both sides; accumulator register v of lane l is row 4 (l / 16) + v and
//    column l % 16 of the block.
//  * No LDS on the way in: a lane loads its 16 bytes of a row as they lie, so a load
//    instruction reads 64 bytes of each of 16 rows and U of them whole lines. The next panel
//    is loaded before this one is multiplied. Rows off a word's boundary (ALIGNED false) are
//    loaded by words and moved into place (load_words).
//  * Rows past M and columns past N repeat the last one; their sums are not stored. Chunks
//    past K are zero (load_tail).
// Bound by reading B: 1 x 8192 x 8192 takes 13.6 us (4.9 TB/s with the launch) at 1 x 1 blocks and
// panels of 256; before its scales were loaded first 14.1, and beside that panels of 512 17.1, 2 column blocks 19.3, the tile kernel at 64 x 64 20.7. Rows
// off a word's boundary: 17.9 with 2 column blocks and panels of 128, 18.5 with 1.
template <int RB_, int CB_, int WAVES_, int U_, bool ALIGNED_> struct I8Rows {
    static constexpr int RB = RB_, CB = CB_, WAVES = WAVES_, U = U_;
    static constexpr bool ALIGNED = ALIGNED_;
    static constexpr int BM = 16 * RB, BN = 16 * CB, NT = 64 * WAVES, PANEL = 64 * U;
};

template <typename T>
__global__ __launch_bounds__(T::NT) void k_gemm_i8_rows(I8Args p)
{
    __shared__ int sums[T::BM * T::BN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = p.tiles_m * p.tiles_n;
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    const int k0 = split * p.k_chunk, kn = min(p.K - k0, p.k_chunk);
    const int8_t *A = p.A + int64_t(m0) * p.lda + k0;
    const int8_t *B = p.B + int64_t(n0) * p.ldb + k0;
    // a thread stores one element of the tile at most: its scales and bias are loaded now, not behind
    // the sums (1 x 8192 x 8192 14.2 to 13.6 us)
    static_assert(T::BM * T::BN <= T::NT, "an element to a thread");
    const int em = m0 + tid / T::BN, en = n0 + tid % T::BN;
    const bool stores = tid < T::BM * T::BN && em < p.M && en < p.N;
    float esa = 0.0f, esb = 0.0f, ebias = 0.0f;
    if (stores) {
        esa = p.sa[em];
        esb = p.sb[en];
        if (p.bias) ebias = p.bias[en];
    }
    if (tid < T::BM * T::BN) sums[tid] = 0;

    const int r = lane & 15, q = lane >> 4;
    const uint32_t a_low = T::ALIGNED ? 0 : uint32_t(reinterpret_cast<uintptr_t>(A)) & 3;
    const uint32_t b_low = T::ALIGNED ? 0 : uint32_t(reinterpret_cast<uintptr_t>(B)) & 3;
    const int8_t *Aw = A - a_low, *Bw = B - b_low;     // from a word's boundary
    uint32_t ao[T::RB], bo[T::CB];                     // this lane's chunks from there
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
        ao[i] = a_low + uint32_t(min(16 * i + r, p.M - 1 - m0)) * uint32_t(p.lda) + 16 * q;
#pragma unroll
    for (int j = 0; j < T::CB; ++j)
        bo[j] = b_low + uint32_t(min(16 * j + r, p.N - 1 - n0)) * uint32_t(p.ldb) + 16 * q;

    i32x4 acc[T::RB][T::CB];
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
#pragma unroll
        for (int j = 0; j < T::CB; ++j) acc[i][j] = i32x4(0);
    struct Aligned {
        i32x4 body;
    };
    typedef std::conditional_t<T::ALIGNED, Aligned, Unaligned> Chunk;
    struct Panel {
        Chunk a[T::U][T::RB], b[T::U][T::CB];
    };
    auto fetch = [&](const int8_t *base, uint32_t off) __attribute__((always_inline)) {
        if constexpr (T::ALIGNED) return Chunk{*reinterpret_cast<const i32x4 *>(base + off)};
        else return load_words(base, off & ~3u, (off + 15) & ~3u);
    };
    auto value = [&](const Chunk &c, uint32_t off) __attribute__((always_inline)) {
        if constexpr (T::ALIGNED) return c.body;
        else return join_words(c, off);
    };
    auto load = [&](Panel &x, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < T::U; ++u)
#pragma unroll
            for (int j = 0; j < T::CB; ++j) x.b[u][j] = fetch(Bw + k + 64 * u, bo[j]);
#pragma unroll
        for (int u = 0; u < T::U; ++u)
#pragma unroll
            for (int i = 0; i < T::RB; ++i) x.a[u][i] = fetch(Aw + k + 64 * u, ao[i]);
    };
    auto multiply = [&](const Panel &x) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < T::U; ++u) {
            i32x4 a[T::RB];
#pragma unroll
            for (int i = 0; i < T::RB; ++i) a[i] = value(x.a[u][i], ao[i]);
#pragma unroll
            for (int j = 0; j < T::CB; ++j) {
                const i32x4 b = value(x.b[u][j], bo[j]);
#pragma unroll
                for (int i = 0; i < T::RB; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b, acc[i][j], 0, 0, 0);
            }
        }
    };
    constexpr int STRIDE = T::WAVES * T::PANEL;
    const int whole = kn / T::PANEL * T::PANEL;        // end of the whole panels
    const int first = wave * T::PANEL;
    if (first < whole) {
        Panel x;
        load(x, first);
#pragma unroll 2
        for (int k = first + STRIDE; k < whole; k += STRIDE) {
            Panel y;
            load(y, k);
            __builtin_amdgcn_sched_barrier(0);
            multiply(x);
            x = y;
        }
        multiply(x);
    }
    // what is left of K, less than a panel, in steps of 64 by the waves in turn
    for (int t = whole + 64 * wave; t < kn; t += 64 * T::WAVES) {
        i32x4 a[T::RB], b[T::CB];
#pragma unroll
        for (int i = 0; i < T::RB; ++i) a[i] = load_tail(Aw + ao[i] - 16 * q, t + 16 * q, kn);
#pragma unroll
        for (int j = 0; j < T::CB; ++j) b[j] = load_tail(Bw + bo[j] - 16 * q, t + 16 * q, kn);
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int j = 0; j < T::CB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }

    __syncthreads();
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
#pragma unroll
        for (int j = 0; j < T::CB; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                __hip_atomic_fetch_add(&sums[(16 * i + 4 * q + v) * T::BN + 16 * j + r],
                                       acc[i][j][v], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
    __syncthreads();
    if (!stores) return;
    if (p.splits > 1) {
        p.partial[(int64_t(split) * p.M + em) * p.N + en] = sums[tid];
        return;
    }
    const float x[1] = {i8_value(sums[tid], esa, esb, ebias)};
    i8_store_as<1>(p.c_dtype, p.C, em * p.ldc + en, x, 1);
}

}  // namespace sgemm
