// byte_tiles.hpp -- what the products of 8-bit and of 4-bit operands share: tiles whose operands are
// rows of bytes, their way into LDS, rows off a word's boundary, and stores of C.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernel_mfma.hpp"
#include "ops_common.hpp"

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ stores of C ---------
template <int DT, int W, bool STREAM = false>
__device__ inline void store_values(void *C, int64_t at, const float (&v)[W], int valid)
{
    typedef typename Elem<DT>::type T;
    T *c = static_cast<T *>(C) + at;
    if (valid >= W) {
        Pack<T, W> p;
#pragma unroll
        for (int j = 0; j < W; ++j) p.v[j] = Elem<DT>::narrow(v[j]);
        if constexpr (STREAM) store_pack_stream(c, p);
        else store_pack(c, p);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < valid) c[j] = Elem<DT>::narrow(v[j]);
    }
}

template <int W>
__device__ inline void store_values_as(int dtype, void *C, int64_t at, const float (&v)[W], int valid)
{
    if (dtype == SGEMM_DTYPE_BF16) store_values<SGEMM_DTYPE_BF16, W>(C, at, v, valid);
    else if (dtype == SGEMM_DTYPE_F16) store_values<SGEMM_DTYPE_F16, W>(C, at, v, valid);
    else store_values<SGEMM_DTYPE_F32, W>(C, at, v, valid);
}

// ------------------------------------------------------------------ tiles ---------------
// A BM x BN tile of C by WGM x WGN waves, BK bytes of each row of both operands at a time, NSTG of
// those panels in LDS. An MFMA takes 32 x 32 of C and 32 bytes of a row.
template <int BM_, int BN_, int WGM_, int WGN_, int BK_, int NSTG_> struct ByteTile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, BK = BK_, NSTG = NSTG_;
    static constexpr int NT = 64 * WGM * WGN;
    static constexpr int WM = BM / WGM, WN = BN / WGN;
    static constexpr int RB = WM / 32, CB = WN / 32;
    static constexpr int CPR = BK / 16;              // chunks per row
    static constexpr int STEPS = BK / 32;            // MFMA steps per panel
    static constexpr int ACH = BM * CPR / NT, BCH = BN * CPR / NT;   // chunks per thread
    static constexpr int A_BYTES = BM * BK, STAGE = (BM + BN) * BK;
    // one workgroup to a compute unit: it goes on to another tile
    static constexpr bool LOOP = NSTG * STAGE > 80 * 1024;
    static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0, "whole chunks per thread");
    static_assert(NT / CPR % a_swizzle_period<CPR>() == 0, "one swizzle per thread");
};

// Global row of B (within the tile) at LDS row p.
template <typename T> __device__ inline int tile_b_row(int p)
{
    const int w = p / T::WN, r = p % T::WN;
    return w * T::WN + T::CB * (r % 32) + r / 32;
}

// Size of the resource that covers [from, end), `end` rounded up to a whole word.
__device__ inline uint32_t bytes_range(const int8_t *from, const int8_t *end)
{
    const int64_t n = end - from;
    return n <= 0 ? 0u : n >= int64_t(kFullRange) ? kFullRange : (uint32_t(n) + 3u) & ~3u;
}

// 16 bytes a lane from base + off, zeros where that is past `range`, to LDS at `to` + 16 lanes.
typedef __attribute__((address_space(3))) void *lds_ptr;
__device__ __forceinline__ void load16_lds(const int8_t *base, uint32_t range, uint32_t off, char *to)
{
    const auto rsrc = make_rsrc32(reinterpret_cast<const float *>(base), range);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)to, 16, off, 0, 0, 0);
}

// 64 floats from base + first to LDS, at `to` + 4 lanes: zeros from `count` on.
__device__ __forceinline__ void load_floats_lds(const float *base, int first, int count, int lane, char *to)
{
    const auto rsrc = make_rsrc32(base, uint32_t(max(count, 0)) * 4u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)to, 4, (first + lane) * 4, 0, 0, 0);
}

// The tile of workgroup bid, in tile_coords' order. Divisions by numbers the host knows are a
// product's upper half and a shift there (exact below 2^31): a division takes some 200 cycles that
// nothing covers at a kernel's start.
template <typename Args> __device__ inline void tile_of(const Args &p, int bid, int &tm, int &tn)
{
    const int t = xcd_contiguous(bid, p.tiles_m * p.tiles_n);
    const int g = int(__umulhi(uint32_t(t), p.group_mul) >> p.group_shift);
    const int w = t - g * kGroupM * p.tiles_n, first = g * kGroupM;
    const int rows = min(p.tiles_m - first, kGroupM);
    static_assert(kGroupM == 8, "whole groups are divided by shifts");
    if (rows == kGroupM) {
        tm = first + w % kGroupM;
        tn = w / kGroupM;
    } else {
        tm = first + w % rows;
        tn = w / rows;
    }
}

// ---- rows of any alignment
// 16 bytes at any address from the aligned words that hold them: four words from the one
// that holds the first byte, and the one that holds the last.
struct Unaligned {
    i32x4 body;
    int last;
};
__device__ inline Unaligned load_words(const int8_t *base, uint32_t first, uint32_t last)
{
    return {*reinterpret_cast<const i32x4 *>(base + first), *reinterpret_cast<const int *>(base + last)};
}
// Moves them into place; the low two bits of `shift` are the address's.
__device__ inline i32x4 join_words(const Unaligned &w, uint32_t shift)
{
    return i32x4{int(__builtin_amdgcn_alignbyte(w.body[1], w.body[0], shift)),
                 int(__builtin_amdgcn_alignbyte(w.body[2], w.body[1], shift)),
                 int(__builtin_amdgcn_alignbyte(w.body[3], w.body[2], shift)),
                 int(__builtin_amdgcn_alignbyte(w.last, w.body[3], shift))};
}
// The first `left` of 16 bytes, zeros behind them.
__device__ inline i32x4 keep_bytes(i32x4 v, int left)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        v[i] = n >= 4 ? v[i] : n <= 0 ? 0 : v[i] & ((1 << 8 * n) - 1);
    }
    return v;
}

// The chunk of 16 bytes at k of a row that ends at kn, which the chunk may cross or lie past:
// zeros from there on, and no byte past kn is read. A row of 16 bytes and more is read at
// its last 16, which are moved into place.
__device__ inline i32x4 load_tail(const int8_t *row, int k, int kn)
{
    unsigned __int128 v = 0;
    if (k < kn) {
        if (kn >= 16) {
            const int at = min(k, kn - 16);
            const Pack<int, 4> w = load_pack<int, 4>(reinterpret_cast<const int *>(row + at));
            v = __builtin_bit_cast(unsigned __int128, w) >> (8 * (k - at));
        } else {
            for (int e = kn - 1; e >= k; --e) v = v << 8 | uint8_t(row[e]);
        }
    }
    return __builtin_bit_cast(i32x4, v);
}

// ------------------------------------------------------------------ rows put in place ---
// Copies rows of any length and alignment to rows of whole 16-byte chunks, zeros behind
// their ends, for products large enough to earn it. A workgroup copies `rows` rows at a time
// (about 2048 chunks).
struct Rows16 {
    const int8_t *src;
    int8_t *dst;
    int64_t ld;
    int count, rows, blocks;     // rows in all, rows to a workgroup, workgroups
};

// One workgroup's share (256 threads), `block` of p.blocks: rows of K bytes.
__device__ inline void put_rows_in_place(const Rows16 &p, int block, int K)
{
    const int cpr = (K + 15) / 16;
    const int64_t row0 = int64_t(block) * p.rows;
    const int n = min(p.rows, int(p.count - row0)) * cpr;
    const int8_t *src = p.src + row0 * p.ld;
    i32x4 *dst = reinterpret_cast<i32x4 *>(p.dst) + row0 * cpr;
    constexpr int U = 4;
    for (int e0 = threadIdx.x; e0 < n; e0 += 256 * U) {
        Unaligned w[U];
        uint32_t low[U];
        int left[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = min(e0 + 256 * u, n - 1);
            const int r = e / cpr, k = (e - r * cpr) * 16;
            const int8_t *row = src + r * p.ld;
            left[u] = K - k;
            low[u] = uint32_t(reinterpret_cast<uintptr_t>(row + k)) & 3;
            if (left[u] >= 16) w[u] = load_words(row + k - low[u], 0, (low[u] + 15) & ~3u);
            else w[u] = {load_tail(row, k, K), 0};
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (e0 + 256 * u < n)
                dst[e0 + 256 * u] = left[u] >= 16 ? join_words(w[u], low[u]) : w[u].body;
    }
}


}  // namespace sgemm
