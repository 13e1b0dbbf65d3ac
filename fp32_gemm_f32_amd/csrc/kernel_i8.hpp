// kernel_i8.hpp -- kernels of the 8-bit product (gemm_i8.h): the tile kernel on
// v_mfma_i32_32x32x32_i8, the join of its split form, and the row quantiser.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernel_mfma.hpp"
#include "ops_common.hpp"

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct I8Args {
    const int8_t *A;
    const int8_t *B;
    const float *sa;
    const float *sb;
    const float *bias;     // or NULL
    void *C;
    int *partial;          // splits > 1: sums of split s at partial + s * M * N
    int64_t lda, ldb, ldc;
    int M, N, K;
    int c_dtype;
    int tiles_m, tiles_n;
    uint32_t group_mul;    // division by kGroupM * tiles_n without dividing: see i8_tile
    int group_shift;
    int splits, k_chunk;   // split s covers k in [s * k_chunk, min(K, (s + 1) * k_chunk))
    bool stream;           // C's rows start on lines of 64 bytes: store past the caches
};

// C's value from the exact integer sum: one rounding to FP32, one of the scales' product, and one
// of both the scaling and the bias, said outright so that every kernel's are the same bits whatever
// the compiler may contract.
__device__ inline float i8_value(int sum, float sa, float sb, float bias)
{
    return __builtin_fmaf(static_cast<float>(sum), sa * sb, bias);
}

template <int DT, int W, bool STREAM = false>
__device__ inline void i8_store(void *C, int64_t at, const float (&v)[W], int valid)
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
__device__ inline void i8_store_as(int dtype, void *C, int64_t at, const float (&v)[W], int valid)
{
    if (dtype == SGEMM_DTYPE_BF16) i8_store<SGEMM_DTYPE_BF16, W>(C, at, v, valid);
    else if (dtype == SGEMM_DTYPE_F16) i8_store<SGEMM_DTYPE_F16, W>(C, at, v, valid);
    else i8_store<SGEMM_DTYPE_F32, W>(C, at, v, valid);
}

// ------------------------------------------------------------------ the tile kernel ----
//
// One workgroup computes a BM x BN tile with WGM x WGN waves of (BM / WGM) x (BN / WGN),
// panel by panel of BK bytes of K.
//  * A panel's rows are BK / 16 chunks of 16 bytes; chunk q of row r lies at chunk
//    position q ^ a_swizzle(r), so the 32 rows that one ds_read_b128 of an MFMA operand
//    reads lie on distinct banks.
//  * MFMA operands (32x32x32): lane l supplies row l % 32 and 16 values of k, the chunk
//    2 t + l / 32 of step t, on both sides. Accumulator register v of lane l is row
//    8 (v / 4) + v % 4 + 4 (l / 32) and column l % 32 of the block.
//  * A lane's CB column blocks are consecutive columns of C: LDS row 32 j + c of a wave's
//    share of B holds global row CB c + j, so lane column c of block j is column CB c + j
//    and one store writes CB neighbours.
//  * Loads go straight to LDS (buffer loads, 16 bytes a lane), NSTG panels deep; chunks past
//    the tile's rows or past K read as zero through an offset out of range. That needs rows
//    on word boundaries and K a multiple of 16.
//  * ANY takes rows at any address and any K. Loads start at the word that holds a row's
//    first byte, so a row lies in LDS off its place by its address's low two bits. An operand
//    is read with the word behind it, which may be the next panel's first, and moved into
//    place (join_words) before it is multiplied. In the panel that holds K's end A's
//    values past it are zeroed there, so B's do not count. Words are loaded only where one
//    of their bytes may be the matrix's (the resource ends with its last row).
// Large products are bound by power: 8192^3 to bf16 takes 442 us once the clock has settled (2490
// TOP/s; 497 over a process's first launches) with the matrix pipes busy 75 % of the cycles at 1.59 GHz. Small ones by the latency of
// a start, the first panels and the stores (1024^3 5.5 us), few rows by reading B (48 x 16384 x
// 4096 13.0 us, 5.1 TB/s).
template <int BM_, int BN_, int WGM_, int WGN_, int BK_, int NSTG_> struct I8Tile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, BK = BK_, NSTG = NSTG_;
    static constexpr int NT = 64 * WGM * WGN;
    static constexpr int WM = BM / WGM, WN = BN / WGN;
    static constexpr int RB = WM / 32, CB = WN / 32;
    static constexpr int CPR = BK / 16;              // chunks per row
    static constexpr int STEPS = BK / 32;            // MFMA steps per panel
    static constexpr int ACH = BM * CPR / NT, BCH = BN * CPR / NT;   // chunks per thread
    static constexpr int A_BYTES = BM * BK, STAGE = (BM + BN) * BK;
    static constexpr int SN = (BN + 63) / 64 * 64;   // floats B's scales take in LDS, and the bias
    // one workgroup to a compute unit: it goes on to another tile
    static constexpr bool LOOP = NSTG * STAGE > 80 * 1024;
    static_assert(BM % 64 == 0, "A's scales are loaded 64 at a time");
    static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0, "whole chunks per thread");
    static_assert(NT / CPR % a_swizzle_period<CPR>() == 0, "one swizzle per thread");
};

// Global row of B (within the tile) at LDS row p.
template <typename T> __device__ inline int i8_b_row(int p)
{
    const int w = p / T::WN, r = p % T::WN;
    return w * T::WN + T::CB * (r % 32) + r / 32;
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

// Stores a wave's accumulators (or, in the split form, its sums): this lane's rows
// 8 (v / 4) + v % 4 + 4 (l / 32) of each row block, columns CB (l % 32) + 0 .. CB - 1 of the
// wave's share.
template <typename T>
__device__ __forceinline__ void i8_epilogue(const I8Args &p, const i32x16 (&acc)[T::RB][T::CB],
                                            const float *scales, int m0, int n0, int split, int wm,
                                            int wn)
{
    const int frow = threadIdx.x & 31, fhi = (threadIdx.x & 63) >> 5;
    const int col = n0 + wn * T::WN + T::CB * frow;
    const int valid = p.N - col;
    const int row0 = m0 + wm * T::WM + 4 * fhi;
    if (valid <= 0) return;
    if (p.splits > 1) {
        int *out = p.partial + int64_t(split) * p.M * p.N;
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int m = row0 + 32 * i + 8 * (v / 4) + v % 4;
                if (m < p.M)
#pragma unroll
                    for (int j = 0; j < T::CB; ++j)
                        if (j < valid) out[int64_t(m) * p.N + col + j] = acc[i][j][v];
            }
        return;
    }
    // the scales and the bias wait in LDS: A's of the tile's rows, B's of its columns, the bias
    float sa[T::RB][16], sb[T::CB], bias[T::CB];
    const float *sbs = scales + T::BM + wn * T::WN + T::CB * frow;
#pragma unroll
    for (int j = 0; j < T::CB; ++j) {
        sb[j] = sbs[j];
        bias[j] = p.bias ? sbs[T::SN + j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) sa[i][v] = scales[wm * T::WM + 4 * fhi + 32 * i + 8 * (v / 4) + v % 4];
    auto store_all = [&](auto dt, auto stream) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int m = row0 + 32 * i + 8 * (v / 4) + v % 4;
                float x[T::CB];
#pragma unroll
                for (int j = 0; j < T::CB; ++j) x[j] = i8_value(acc[i][j][v], sa[i][v], sb[j], bias[j]);
                if (m < p.M)
                    i8_store<decltype(dt)::value, T::CB, decltype(stream)::value>(p.C, m * p.ldc + col, x, valid);
            }
    };
    auto store = [&](auto dt) __attribute__((always_inline)) {
        if (p.stream) store_all(dt, std::true_type{});
        else store_all(dt, std::false_type{});
    };
    if (p.c_dtype == SGEMM_DTYPE_BF16) store(std::integral_constant<int, SGEMM_DTYPE_BF16>{});
    else if (p.c_dtype == SGEMM_DTYPE_F16) store(std::integral_constant<int, SGEMM_DTYPE_F16>{});
    else store(std::integral_constant<int, SGEMM_DTYPE_F32>{});
}

// Size of the resource that covers [from, end), `end` rounded up to a whole word.
__device__ inline uint32_t i8_range(const int8_t *from, const int8_t *end)
{
    const int64_t n = end - from;
    return n <= 0 ? 0u : n >= int64_t(kFullRange) ? kFullRange : (uint32_t(n) + 3u) & ~3u;
}

// 16 bytes a lane from base + off, zeros where that is past `range`, to LDS at `to` + 16 lanes.
typedef __attribute__((address_space(3))) void *lds_ptr;
__device__ __forceinline__ void i8_load16_lds(const int8_t *base, uint32_t range, uint32_t off, char *to)
{
    const auto rsrc = make_rsrc32(reinterpret_cast<const float *>(base), range);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)to, 16, off, 0, 0, 0);
}

// 64 floats from base + first to LDS, at `to` + 4 lanes: zeros from `count` on.
__device__ __forceinline__ void i8_load_floats(const float *base, int first, int count, int lane, char *to)
{
    const auto rsrc = make_rsrc32(base, uint32_t(max(count, 0)) * 4u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)to, 4, (first + lane) * 4, 0, 0, 0);
}

// The tile of workgroup bid, in tile_coords' order. Divisions by numbers the host knows are a
// product's upper half and a shift there (exact below 2^31): a division takes some 200 cycles that
// nothing covers at a kernel's start.
__device__ inline void i8_tile(const I8Args &p, int bid, int &tm, int &tn)
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

template <typename T, bool ANY>
__global__ __launch_bounds__(T::NT) void k_gemm_i8(I8Args p)
{
    constexpr int STAGE = T::STAGE;
    constexpr int SCALES = (T::BM + 2 * T::SN) * 4;
    constexpr bool LOOP = T::LOOP && !ANY;
    static_assert(T::NSTG >= 2 && T::NSTG * STAGE + (LOOP ? 2 : 1) * SCALES <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(16))) char smem[T::NSTG * STAGE + (LOOP ? 2 : 1) * SCALES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / T::WGN, wn = wave % T::WGN;
    const int tiles = p.tiles_m * p.tiles_n;
    const int split = p.splits == 1 ? 0 : int(blockIdx.x) / tiles;
    const int k0 = split * p.k_chunk, k1 = min(p.K, k0 + p.k_chunk);
    const int panels = (k1 - k0 + T::BK - 1) / T::BK;
    const int kn = k1 - k0;                          // values of k in this split

    // the tile that loads go to: this thread's chunks, LDS chunk i * NT + tid
    const int prow = tid / T::CPR;                   // LDS row of chunk i = 0
    const int q = (tid % T::CPR) ^ a_swizzle<T::CPR>(prow);
    int m0, n0;
    const int8_t *At, *Bt;
    uint32_t a_low = 0, b_low = 0, a_off[T::ACH], b_off[T::BCH];
    auto aim = [&](int tile) __attribute__((always_inline)) {
        int tm, tn;
        i8_tile(p, tile, tm, tn);
        m0 = tm * T::BM;
        n0 = tn * T::BN;
        At = p.A + m0 * p.lda + k0;
        Bt = p.B + n0 * p.ldb + k0;
        if constexpr (ANY) {
            a_low = uint32_t(reinterpret_cast<uintptr_t>(At)) & 3;
            b_low = uint32_t(reinterpret_cast<uintptr_t>(Bt)) & 3;
            At -= a_low;
            Bt -= b_low;
        }
#pragma unroll
        for (int i = 0; i < T::ACH; ++i) {
            const int r = prow + i * (T::NT / T::CPR);
            a_off[i] = m0 + r < p.M ? (a_low + uint32_t(r * p.lda) + q * 16) & ~3u : kOob;
        }
#pragma unroll
        for (int i = 0; i < T::BCH; ++i) {
            const int r = i8_b_row<T>(prow + i * (T::NT / T::CPR));
            b_off[i] = n0 + r < p.N ? (b_low + uint32_t(r * p.ldb) + q * 16) & ~3u : kOob;
        }
    };
    int tile = int(blockIdx.x) - split * tiles;
    aim(tile);
    i32x16 acc[T::RB][T::CB];
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
#pragma unroll
        for (int j = 0; j < T::CB; ++j) acc[i][j] = i32x16(0);

    // operand reads: row l % 32 of a block; chunk 2 t + l / 32 at step t, with ANY t + STEPS (l / 32),
    // so that the word behind a lane's chunk is the first of its own next one (any order of k
    // does that is the same on both sides)
    const int frow = lane & 31, fhi = lane >> 5;
    const int fsw = a_swizzle<T::CPR>(frow);
    const int a_row = wm * T::WM + frow, b_row = wn * T::WN + frow;
    const int a_base = a_row * T::BK, b_base = T::A_BYTES + b_row * T::BK;
    i32x4 fa[T::STEPS][T::RB], fb[T::STEPS][T::CB];
    // ANY: the words behind the last step's chunks: of lanes below 32 the panel's chunk STEPS, of
    // the others the next panel's first
    int na[2][T::RB], nb[2][T::CB];
    uint32_t a_shift[T::RB], b_shift[T::CB];
    if constexpr (ANY) {
#pragma unroll
        for (int i = 0; i < T::RB; ++i) a_shift[i] = a_low + uint32_t(a_row + 32 * i) * uint32_t(p.lda);
#pragma unroll
        for (int j = 0; j < T::CB; ++j)
            b_shift[j] = b_low + uint32_t(i8_b_row<T>(b_row + 32 * j)) * uint32_t(p.ldb);
    }
    auto read = [&](const char *st, auto tc) __attribute__((always_inline)) {
        constexpr int t = decltype(tc)::value;
        const int at = ((ANY ? t + T::STEPS * fhi : 2 * t + fhi) ^ fsw) * 16;
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
            fa[t][i] = *reinterpret_cast<const i32x4 *>(st + a_base + at + i * 32 * T::BK);
#pragma unroll
        for (int j = 0; j < T::CB; ++j)
            fb[t][j] = *reinterpret_cast<const i32x4 *>(st + b_base + at + j * 32 * T::BK);
        if constexpr (ANY && (t == T::STEPS - 1 || t == 0)) {
            const int behind = ((t == 0 ? 0 : T::STEPS) ^ fsw) * 16;
            constexpr int of = t == 0 ? 1 : 0;
#pragma unroll
            for (int i = 0; i < T::RB; ++i)
                na[of][i] = *reinterpret_cast<const int *>(st + a_base + behind + i * 32 * T::BK);
#pragma unroll
            for (int j = 0; j < T::CB; ++j)
                nb[of][j] = *reinterpret_cast<const int *>(st + b_base + behind + j * 32 * T::BK);
        }
    };
    // MASK: values of k from `left` on (of this lane's chunk) count as zero
    auto multiply = [&](auto tc, auto mask, int left) __attribute__((always_inline)) {
        constexpr int t = decltype(tc)::value, u = t + 1 < T::STEPS ? t + 1 : t;
        if constexpr (ANY) {
#pragma unroll
            for (int i = 0; i < T::RB; ++i) {
                fa[t][i] = join_words({fa[t][i], u > t ? fa[u][i][0] : fhi ? na[1][i] : na[0][i]}, a_shift[i]);
                if constexpr (decltype(mask)::value) fa[t][i] = keep_bytes(fa[t][i], left);
            }
#pragma unroll
            for (int j = 0; j < T::CB; ++j)
                fb[t][j] = join_words({fb[t][j], u > t ? fb[u][j][0] : fhi ? nb[1][j] : nb[0][j]}, b_shift[j]);
        }
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int j = 0; j < T::CB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[t][i], fb[t][j], acc[i][j], 0, 0, 0);
    };

    const int8_t *const a_end = p.A + (p.M - 1) * p.lda + p.K, *const b_end = p.B + (p.N - 1) * p.ldb + p.K;
    auto issue = [&](int panel, char *st) __attribute__((always_inline)) {
        const int k = panel * T::BK;
        const int8_t *const ak = At + k, *const bk = Bt + k;
        const uint32_t an = ANY ? i8_range(ak, a_end) : kFullRange;
        const uint32_t bn = ANY ? i8_range(bk, b_end) : kFullRange;
        // in the range's last panel, and past it, chunks past its end read as zero (a row
        // that lies off its place by up to 3 bytes may end in the next chunk)
        const uint32_t past = k + q * 16 >= kn + (ANY ? 3 : 0) ? kOob : 0u;
#pragma unroll
        for (int i = 0; i < T::ACH; ++i)
            i8_load16_lds(ak, an, a_off[i] | past, st + (i * T::NT + wave * 64) * 16);
#pragma unroll
        for (int i = 0; i < T::BCH; ++i)
            i8_load16_lds(bk, bn, b_off[i] | past, st + T::A_BYTES + (i * T::NT + wave * 64) * 16);
    };
    // Operands are read LOOK steps ahead. LOOK steps before a panel's end the reads of its stage
    // are over, so the barrier comes there: the wave's loads of the next panel have landed, every
    // wave's have after the barrier, and the stage just read is loaded again and the next one's
    // first operands are read under the last steps' MFMAs.
    constexpr int LPP = T::ACH + T::BCH;
    constexpr int LOOK = ANY ? 2 : 1;
    // ahead of the panels, so that the first wait covers them: the epilogue's scales and bias (1024^3
    // 6.2 to 5.7 us against loading them there)
    char *scales = smem + T::NSTG * STAGE;
    auto issue_scales = [&](char *at_lds) __attribute__((always_inline)) {
        for (int i = wave; p.splits == 1 && i < (T::BM + 2 * T::SN) / 64; i += T::NT / 64) {
            char *to = at_lds + i * 256;
            const int at = i * 64;
            if (at < T::BM) i8_load_floats(p.sa + m0, at, min(p.M - m0, T::BM), lane, to);
            else if (at < T::BM + T::SN) i8_load_floats(p.sb + n0, at - T::BM, min(p.N - n0, T::BN), lane, to);
            else if (p.bias) i8_load_floats(p.bias + n0, at - T::BM - T::SN, min(p.N - n0, T::BN), lane, to);
        }
    };
    issue_scales(scales);
#pragma unroll
    for (int i = 0; i < T::NSTG; ++i) issue(i, smem + i * STAGE);
    wait_vmcnt<(T::NSTG - 1) * LPP>();
    asm volatile("s_barrier" ::: "memory");
    static_for<0, LOOK>([&](auto tc) __attribute__((always_inline)) { read(smem, tc); });
    int stage = 0;
    const int full = ANY ? kn / T::BK : panels;      // panels without a masked step
    int behind = 0;                                  // panels between a panel read and that of its tile
    auto run = [&](int panel, auto mask) __attribute__((always_inline)) {
        char *st = smem + stage * STAGE;
        stage = stage + 1 == T::NSTG ? 0 : stage + 1;
        const char *next = smem + stage * STAGE;
        static_for<0, T::STEPS>([&](auto tc) __attribute__((always_inline)) {
            constexpr int t = decltype(tc)::value;
            constexpr bool turn = t == T::STEPS - LOOK;
            if constexpr (turn) {
                __builtin_amdgcn_sched_barrier(0);
                wait_vmcnt<(T::NSTG - 2) * LPP>();
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            }
            if constexpr (t + LOOK < T::STEPS) read(st, std::integral_constant<int, t + LOOK>{});
            else read(next, std::integral_constant<int, t + LOOK - T::STEPS>{});
            if constexpr (turn) issue(panel + T::NSTG - behind, st);
            multiply(tc, mask, kn - panel * T::BK - 16 * (ANY ? t + T::STEPS * fhi : 2 * t + fhi));
            // operand reads behind the first MFMAs, the loads behind the others
            constexpr int ops = (T::RB + T::CB) * (ANY && (t + LOOK) % T::STEPS % (T::STEPS - 1) == 0 ? 2 : 1);
            constexpr int mf = T::RB * T::CB;
            constexpr int rm = turn ? (mf + 1) / 2 : (ops < mf ? ops : mf);
            constexpr int lm = mf - rm > 0 ? mf - rm : 1;
            static_for<0, mf>([&](auto mc) __attribute__((always_inline)) {
                constexpr int m = decltype(mc)::value;
                constexpr int r = m < rm ? (m + 1) * ops / rm - m * ops / rm : 0;
                constexpr int n = m - (mf - lm);
                constexpr int l = turn && n >= 0 ? (n + 1) * LPP / lm - n * LPP / lm : 0;
                __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
                if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(kSchedDsRead, r, 0);
                if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(kSchedVmemRead, l, 0);
            });
        });
    };
    if constexpr (!LOOP) {
        for (int panel = 0; panel < full; ++panel) run(panel, std::false_type{});
        if constexpr (ANY)
            if (full < panels) run(full, std::true_type{});
        wait_vmcnt<0>();   // no load is in flight to LDS when the workgroup ends
        i8_epilogue<T>(p, acc, reinterpret_cast<const float *>(scales), m0, n0, split, wm, wn);
    } else {
        // The last NSTG panels of a tile load the first of the next, so that its stores and the start
        // of the next run under each other: 8192 x 8192 x 256 to bf16 47 to 39 us, x 2048 131 to 124 (the
        // grid has fewer workgroups than tiles only where K has NSTG panels). Not waiting for
        // the stores before the panels behind them gave 1 % at most, and the same for tiles of
        // which two share a compute unit nothing: they overlap as they are.
        for (;;) {
            const int cm0 = m0, cn0 = n0;
            const float *const ready = reinterpret_cast<const float *>(scales);
            tile += int(gridDim.x);
            const bool more = p.splits == 1 && tile < tiles;
            int panel = 0;
            for (int part = 0; part < 2; ++part) {
                const int end = part == 0 ? panels - T::NSTG : panels;
                for (; panel < end; ++panel) run(panel, std::false_type{});
                if (part == 0 && more) {
                    aim(tile);
                    behind = panels;
                    scales = smem + T::NSTG * STAGE + (scales == smem + T::NSTG * STAGE ? SCALES : 0);
                    issue_scales(scales);
                }
            }
            if (!more) wait_vmcnt<0>();
            i8_epilogue<T>(p, acc, ready, cm0, cn0, split, wm, wn);
            if (!more) break;
            behind = 0;
            // the next switch loads scales where this tile's were: a turn, or this, lies between
            if (panels == T::NSTG) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int i = 0; i < T::RB; ++i)
#pragma unroll
                for (int j = 0; j < T::CB; ++j) acc[i][j] = i32x16(0);
        }
    }
}

// ------------------------------------------------------------------ rows put in place ---
// Copies rows of any length and alignment to rows of whole 16-byte chunks, zeros behind
// their ends, for products large enough to earn it. A workgroup copies `rows` rows at a time
// (about 2048 chunks), of A in its first blocks and of B in the others.
struct I8Rows16 {
    const int8_t *src;
    int8_t *dst;
    int64_t ld;
    int count, rows, blocks;     // rows in all, rows to a workgroup, workgroups
};

__global__ __launch_bounds__(256) void k_gemm_i8_align(I8Rows16 a, I8Rows16 b, int K)
{
    const bool of_a = int(blockIdx.x) < a.blocks;
    const I8Rows16 &p = of_a ? a : b;
    const int block = blockIdx.x - (of_a ? 0 : a.blocks);
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

// ------------------------------------------------------------------ the split's join ----
// Adds the splits' integer sums (exact in any order) and applies the epilogue; one thread
// per element of C, strided over the grid. Bound by reading splits * M * N integers, which
// the plan keeps small (it splits products with few tiles).
__global__ __launch_bounds__(256) void k_gemm_i8_join(I8Args p)
{
    const int64_t total = int64_t(p.M) * p.N;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < total;
         e += int64_t(gridDim.x) * 256) {
        const int64_t m = e / p.N;
        const int n = int(e - m * p.N);
        int sum = 0;
        for (int s = 0; s < p.splits; ++s) sum += p.partial[s * total + e];
        const float x[1] = {i8_value(sum, p.sa[m], p.sb[n], p.bias ? p.bias[n] : 0.0f)};
        i8_store_as<1>(p.c_dtype, p.C, m * p.ldc + n, x, 1);
    }
}

// K == 0: the empty sum plus the bias.
__global__ __launch_bounds__(256) void k_gemm_i8_empty(I8Args p)
{
    const int64_t total = int64_t(p.M) * p.N;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < total;
         e += int64_t(gridDim.x) * 256) {
        const int64_t m = e / p.N;
        const int n = int(e - m * p.N);
        const float x[1] = {p.bias ? p.bias[n] : 0.0f};
        i8_store_as<1>(p.c_dtype, p.C, m * p.ldc + n, x, 1);
    }
}

// ------------------------------------------------------------------ the row quantiser ---
// The integer of x under `inverse` = 127 / peak: rint rounds ties to even; what is not a
// number (inf * 0, NaN) becomes 0.
__device__ inline int quantize_one(float x, float inverse)
{
    const float y = __builtin_rintf(x * inverse);
    return y == y ? static_cast<int>(__builtin_fminf(__builtin_fmaxf(y, -127.0f), 127.0f)) : 0;
}

// The scale and the inverse from the row's peak. The division is IEEE's; 127 / peak
// overflows for peaks below 3.8e-37 (0 included), and such a row becomes zeros.
__device__ inline void row_scale(float peak, float &scale, float &inverse)
{
    scale = peak / 127.0f;
    inverse = 127.0f / peak;
    if (__builtin_isinf(inverse)) { scale = 0.0f; inverse = 0.0f; }
}

// max that keeps a NaN, for absolute values: as unsigned integers their bits are in order,
// with the NaNs above infinity
__device__ inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// The largest of LANES neighbouring lanes' values (16 and more: cross-lane moves, then shuffles).
template <int LANES> __device__ inline uint32_t lanes_max(uint32_t x)
{
    const auto moved = [](uint32_t v, auto ctrl) {
        return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x = max(x, moved(x, std::integral_constant<int, 0xb1>{}));                        // lane ^ 1
    x = max(x, moved(x, std::integral_constant<int, 0x4e>{}));                        // lane ^ 2
    x = max(x, moved(x, std::integral_constant<int, 0x141>{}));                       // four of eight
    if constexpr (LANES >= 16) x = max(x, moved(x, std::integral_constant<int, 0x140>{}));
    if constexpr (LANES >= 32) x = max(x, uint32_t(__shfl_xor(int(x), 16)));
    if constexpr (LANES >= 64) x = max(x, uint32_t(__shfl_xor(int(x), 32)));
    return x;
}

// LANES lanes (256: the workgroup) share a row, CH chunks of 16 bytes to a thread: the row is read
// once, into registers, and the peak taken over the lanes (and the waves, in LDS). HBM-bound: M K
// (2 or 4) bytes in and M K out, 8192 x 8192 bf16 in 37 us (5.4 TB/s), 4096 x 16384 f32 in 62 (5.4;
// read twice instead 75). Rows of odd length or address use the same loads (one instruction serves
// any alignment); the chunk that holds the row's end is filled element by element.
template <int DT, int CH, int LANES>
__global__ __launch_bounds__(256) void k_quantize_rows(int M, int K, const void *X, int64_t ldx,
                                                       int8_t *Q, int64_t ldq, float *scales)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    __shared__ uint32_t peaks[4];
    const int tid = threadIdx.x;
    const int in_row = tid % LANES;
    const int64_t row = int64_t(blockIdx.x) * (256 / LANES) + tid / LANES;
    // rows past the last: no lane of a row still in use takes anything from them, and where rows
    // take whole workgroups there are none
    if (LANES < 256 && row >= M) return;
    const T *x = static_cast<const T *>(X) + row * ldx;
    Pack<T, W> c[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (in_row + i * LANES) * W;
        if (k + W <= K) {
            c[i] = load_pack<T, W>(x + k);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) c[i].v[j] = k + j < K ? x[k + j] : T(0.0f);
        }
    }
    uint32_t peak = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) peak = max(peak, abs_bits(Elem<DT>::widen(c[i].v[j])));
    peak = lanes_max<LANES < 64 ? LANES : 64>(peak);
    if constexpr (LANES == 256) {
        if ((tid & 63) == 0) peaks[tid >> 6] = peak;
        __syncthreads();
        peak = max(max(peaks[0], peaks[1]), max(peaks[2], peaks[3]));
    }
    float scale, inverse;
    row_scale(__builtin_bit_cast(float, peak), scale, inverse);
    int8_t *q = Q + row * ldq;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (in_row + i * LANES) * W;
        Pack<int8_t, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) o.v[j] = int8_t(quantize_one(Elem<DT>::widen(c[i].v[j]), inverse));
        if (k + W <= K) {
            store_pack_stream(q + k, o);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (k + j < K) q[k + j] = o.v[j];
        }
    }
    if (in_row == 0) scales[row] = scale;
}

// Rows too long for the registers: one workgroup reads the row twice (the second time from
// the caches, for rows that fit them).
template <int DT>
__global__ __launch_bounds__(1024) void k_quantize_long_rows(int K, const void *X, int64_t ldx,
                                                             int8_t *Q, int64_t ldq, float *scales)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    __shared__ uint32_t peaks[16];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(X) + row * ldx;
    int8_t *q = Q + row * ldq;
    const int chunks = K / W;
    uint32_t peak = 0;
#pragma unroll 4
    for (int i = tid; i < chunks; i += 1024) {
        const Pack<T, W> c = load_pack<T, W>(x + int64_t(i) * W);
#pragma unroll
        for (int j = 0; j < W; ++j) peak = max(peak, abs_bits(Elem<DT>::widen(c.v[j])));
    }
    const int64_t last = int64_t(chunks) * W + tid;       // at most W - 1 elements are left
    if (last < K) peak = max(peak, abs_bits(Elem<DT>::widen(x[last])));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) peak = max(peak, uint32_t(__shfl_xor(int(peak), d)));
    if ((tid & 63) == 0) peaks[tid >> 6] = peak;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) peak = max(peak, peaks[w]);
    float scale, inverse;
    row_scale(__builtin_bit_cast(float, peak), scale, inverse);
#pragma unroll 4
    for (int i = tid; i < chunks; i += 1024) {
        const Pack<T, W> c = load_pack<T, W>(x + int64_t(i) * W);
        Pack<int8_t, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) o.v[j] = int8_t(quantize_one(Elem<DT>::widen(c.v[j]), inverse));
        store_pack_stream(q + int64_t(i) * W, o);
    }
    if (last < K) q[last] = int8_t(quantize_one(Elem<DT>::widen(x[last]), inverse));
    if (tid == 0) scales[row] = scale;
}

}  // namespace sgemm
