// kernel_mx4_tiles.hpp -- the product of microscaled 4-bit operands (gemm_mx4.h) by tiles, on
// v_mfma_scale_f32_16x16x128_f8f6f4.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "byte_tiles.hpp"
#include "kernel_mx4.hpp"

namespace sgemm {

// One workgroup computes a BM x BN tile with WGM x WGN waves, panel by panel of BK = 128 bytes (256
// elements) of K. Operand bytes move as the 8-bit product's do: straight to LDS, 16 bytes a lane, chunk
// q of row r at chunk position q ^ a_swizzle(r), and a lane's CB column blocks are neighbours in C.
//  * MFMA operands: lane l supplies row l % 16 and one block of 32 values with its scale. Step t of a
//    panel takes block t + 2 (l / 16) on both sides (so that the rows that one ds_read_b128 reads lie
//    on distinct banks). Accumulator register v of lane l is row 4 (l / 16) + v and column l % 16 of the
//    block. These 16 x 16 blocks of 128 values do 8 % more for their power than 32 x 32 of 64 (6.8
//    against 6.3 PFLOP/s from registers, random values), and large products are bound by power.
//  * Panels go in pairs, for their scales come 16 bytes to a row, one load of 16 bytes a lane, ahead of
//    the loads of an even panel, into a ring of their own. In rows they lie 16 bytes here and there,
//    each a line of its own for the caches; large products put them pair by pair of panels first.
//    A lane reads all 16 bytes of a row, the four groups of 16 lanes those of four blocks of rows,
//    and exchanges between the groups give each block a panel's scales: 3 reads for 12 blocks and
//    two panels.
//  * Chunks past the tile's rows or past K read as zero through an offset out of range. Scales behind
//    the last block may be anything and are masked: one that is no number would make zeros NaN. K
//    ends on whole chunks on A's side (B's bytes behind K meet zeros): other A are copied first.
//  * The loop has no branch: with one, the compiler moves the MFMAs of all steps behind it.
//  * Rows have to start on word boundaries, of elements and of scales; others are copied first.
// 8192^3 to bf16 takes 243 us with the quantised values of normal ones (4.5 PFLOP/s; MFMAs alone, fed from
// registers, 162 at the clock that power leaves them), 201 of zeros, which draw little. Without loads in
// the loop it takes 219, without the scales' 249 of 270: they are the next bound. 4096^3 39.5 us. The 256 x 256
// tile takes all 256 registers that a wave of eight may have and spills 11 more, reloaded outside the
// loop over panels, once or twice a tile.
template <int BM_, int BN_, int WGM_, int WGN_, int NSTG_>
struct Mx4Tile : ByteTile<BM_, BN_, WGM_, WGN_, 128, NSTG_> {
    typedef ByteTile<BM_, BN_, WGM_, WGN_, 128, NSTG_> Base;
    static constexpr int RB = Base::WM / 16, CB = Base::WN / 16, STEPS = 2;
    static constexpr int SROWS = (BM_ + BN_ + Base::NT - 1) / Base::NT * Base::NT;   // rows of scales, filled up
    static constexpr int SCH = SROWS / Base::NT;     // a thread's chunks of scales
    static constexpr int SBYTES = SROWS * 16, SRING = NSTG_ / 2;
    static constexpr int LDS = NSTG_ * Base::STAGE + SRING * SBYTES;
    static constexpr bool LOOP = LDS > 80 * 1024;    // one workgroup to a compute unit: it goes on to another tile
    static_assert(LDS <= 160 * 1024, "LDS");
    static_assert(NSTG_ % 2 == 0, "panels go in pairs");
    static_assert(Base::NT / Base::CPR % 16 == 0, "a thread's rows at common distances");
    static_assert(BM_ % 64 == 0, "scales of whole waves");
};

// Global row of B (within the tile) at LDS row p.
template <typename T> __device__ inline int mx4_b_row(int p)
{
    const int w = p / T::WN, r = p % T::WN;
    return w * T::WN + T::CB * (r % 16) + r / 16;
}

template <typename T>
__device__ __forceinline__ void mx4_epilogue(const Mx4Args &p, const f32x4 (&acc)[T::RB][T::CB],
                                             const float (&bias)[T::CB], int m0, int n0, int split, int wm, int wn)
{
    const int lane = threadIdx.x & 63;
    const int col = n0 + wn * T::WN + T::CB * (lane & 15);
    const int valid = p.N - col;
    const int row0 = m0 + wm * T::WM + 4 * (lane >> 4);
    if (valid <= 0) return;
    if (p.splits > 1) {
        float *out = p.partial + int64_t(split) * p.M * p.N;
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = row0 + 16 * i + v;
                if (m < p.M)
#pragma unroll
                    for (int j = 0; j < T::CB; ++j)
                        if (j < valid) out[int64_t(m) * p.N + col + j] = acc[i][j][v];
            }
        return;
    }
    auto store_all = [&](auto dt, auto stream) __attribute__((always_inline)) {
        constexpr int DT = decltype(dt)::value, W = DT == SGEMM_DTYPE_F32 && T::CB > 4 ? 4 : T::CB;   // 16 bytes to a store
#pragma unroll
        for (int i = 0; i < T::RB; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = row0 + 16 * i + v;
                if (m >= p.M) continue;
#pragma unroll
                for (int j = 0; j < T::CB; j += W) {
                    float x[W];
#pragma unroll
                    for (int e = 0; e < W; ++e) x[e] = acc[i][j + e][v] + bias[j + e];
                    store_values<DT, W, decltype(stream)::value>(p.C, m * p.ldc + col + j, x, valid - j);
                }
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

// c + a b with the scales' bytes SA and SB
template <int SA, int SB> __device__ __forceinline__ f32x4 mx4_mfma(i32x4 a, i32x4 b, f32x4 c, int sa, int sb)
{
    const i32x8 ax = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 bx = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ax, bx, c, 4, 4, SA, sa, SB, sb);
}

template <typename T>
__global__ __launch_bounds__(T::NT) void k_mx4_tiles(Mx4Args p)
{
    constexpr int STAGE = T::STAGE;
    __shared__ __attribute__((aligned(16))) char smem[T::LDS];
    char *const ring = smem + T::NSTG * STAGE;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / T::WGN, wn = wave % T::WGN;
    const int tiles = p.tiles_m * p.tiles_n;
    const int split = p.splits == 1 ? 0 : int(blockIdx.x) / tiles;
    const int k0 = split * p.chunk, k1 = min(p.KB, k0 + p.chunk);
    const int kn = k1 - k0;
    // (an odd number is filled up where the next tile's panels follow)
    const int panels = ((kn + T::BK - 1) / T::BK + (T::LOOP ? 1 : 0)) & (T::LOOP ? ~1 : ~0);
    const int blocks = (kn + 15) / 16;               // scales to a row in this split

    // the tile that loads go to: this thread's chunks, LDS chunk i * NT + tid, and rows of scales. Rows
    // past the operand's last lie past its resource's end and read as zero; of a thread's rows one
    // offset is held, the others lie at distances that are the same for all.
    const int prow = tid / T::CPR;                   // LDS row of chunk i = 0
    const int q = (tid % T::CPR) ^ a_swizzle<T::CPR>(prow);
    const uint32_t a_off = uint32_t(prow * p.lda) + q * 16, b_off = uint32_t(mx4_b_row<T>(prow) * p.ldb) + q * 16;
    int m0, n0;
    const int8_t *At, *Bt, *St[T::SCH], *s_end[T::SCH];
    uint32_t a_size, b_size, s_off[T::SCH];
    int s_step[T::SCH];                              // from one pair of panels to the next
    auto aim = [&](int tile) __attribute__((always_inline)) {
        int tm, tn;
        tile_of(p, tile, tm, tn);
        m0 = tm * T::BM;
        n0 = tn * T::BN;
        At = reinterpret_cast<const int8_t *>(p.A) + m0 * p.lda + k0;
        Bt = reinterpret_cast<const int8_t *>(p.B) + n0 * p.ldb + k0;
        a_size = bytes_range(At, reinterpret_cast<const int8_t *>(p.A) + (p.M - 1) * p.lda + p.KB);
        b_size = bytes_range(Bt, reinterpret_cast<const int8_t *>(p.B) + (p.N - 1) * p.ldb + p.KB);
#pragma unroll
        for (int i = 0; i < T::SCH; ++i) {
            // rows of A, then of B as they lie in LDS (a wave's are all of one: BM is a multiple of 64)
            const int s0 = i * T::NT + wave * 64, s = s0 + lane;
            const bool of_a = s0 < T::BM;
            const int64_t ld = of_a ? p.ldsa : p.ldsb;
            const int8_t *const from = reinterpret_cast<const int8_t *>(of_a ? p.sa : p.sb);
            s_step[i] = of_a ? p.sa_step : p.sb_step;
            St[i] = from + (of_a ? m0 : n0) * ld + int64_t(k0 / 256) * s_step[i];
            s_end[i] = from + (of_a ? p.sa_bytes : p.sb_bytes);
            s_off[i] = s >= T::BM + T::BN ? kOob : uint32_t((of_a ? s : mx4_b_row<T>(s - T::BM)) * ld);
        }
    };
    int tile = int(blockIdx.x) - split * tiles;
    aim(tile);
    float bias[T::CB];
    auto load_bias = [&](int n) __attribute__((always_inline)) {
        const int col = n + wn * T::WN + T::CB * (lane & 15);
#pragma unroll
        for (int j = 0; j < T::CB; ++j) bias[j] = p.bias && p.splits == 1 ? p.bias[min(col + j, p.N - 1)] : 0.0f;
    };
    f32x4 acc[T::RB][T::CB];
#pragma unroll
    for (int i = 0; i < T::RB; ++i)
#pragma unroll
        for (int j = 0; j < T::CB; ++j) acc[i][j] = f32x4(0.0f);

    // operand reads: row l % 16 of a block; chunk t + 2 (l / 16) at step t
    const int frow = lane & 15, fq = lane >> 4;
    const int fsw = a_swizzle<T::CPR>(frow);
    // (what is the wave's is kept apart from what is the lane's: it needs no vector registers)
    const int a_base = wm * T::WM * T::BK, b_base = T::A_BYTES + wn * T::WN * T::BK;
    const int lane_at[T::STEPS] = {frow * T::BK + ((T::STEPS * fq) ^ fsw) * 16, frow * T::BK + ((1 + T::STEPS * fq) ^ fsw) * 16};
    i32x4 fa[T::STEPS][T::RB], fb[T::STEPS][T::CB];
    // scales: blocks of rows of A, then of B, in fours; the two halves of the four words are two panels'
    constexpr int BLOCKS = T::RB + T::CB, FOURS = (BLOCKS + 3) / 4;
    i32x4 four[FOURS];
    uint32_t sc[2 * FOURS];                          // of the panel multiplied, two blocks to a word
    int s_at[FOURS];
#pragma unroll
    for (int n = 0; n < FOURS; ++n) {
        const int block = min(4 * n + fq, BLOCKS - 1);
        s_at[n] = ((block < T::RB ? wm * T::WM + 16 * block : T::BM + wn * T::WN + 16 * (block - T::RB)) + frow) * 16;
    }
    // A's operands of a step, and half of B's
    auto read_a = [&](int st, auto tc) __attribute__((always_inline)) {
        constexpr int t = decltype(tc)::value;
        const char *const at = smem + ((st + a_base) + lane_at[t]);
#pragma unroll
        for (int i = 0; i < T::RB; ++i) fa[t][i] = *reinterpret_cast<const i32x4 *>(at + i * 16 * T::BK);
    };
    auto read_b = [&](int st, auto tc, auto hc) __attribute__((always_inline)) {
        constexpr int t = decltype(tc)::value, first = decltype(hc)::value * T::CB / 2;
        const char *const at = smem + ((st + b_base) + lane_at[t]);
#pragma unroll
        for (int j = first; j < first + T::CB / 2; ++j) fb[t][j] = *reinterpret_cast<const i32x4 *>(at + j * 16 * T::BK);
    };
    auto read_scales = [&](int entry) __attribute__((always_inline)) {
        const char *at = ring + entry * T::SBYTES;
#pragma unroll
        for (int n = 0; n < FOURS; ++n) four[n] = *reinterpret_cast<const i32x4 *>(at + s_at[n]);
    };
    // The scales of a panel, the even or odd one of the pair read last. Group g of 16 lanes holds block g's
    // 8 and needs two of them of each block: 2 g and 2 g + 1. Exchanging the halves of the wave leaves
    // blocks 0 and 1 in one word, 2 and 3 in another, each with the right word of a block in every
    // other group; exchanging neighbouring groups spreads it to both, and of two blocks' words the
    // right halves make one: bytes 0 and 1 for the first one's steps, 2 and 3 for the other's.
    const uint32_t halves = fq & 1 ? 0x07060302u : 0x05040100u;
    auto take_scales = [&](int panel, auto odd) __attribute__((always_inline)) {
        constexpr int w = decltype(odd)::value ? 2 : 0;
        const int left = blocks - 8 * panel - 2 * fq;
        const uint32_t keep = left >= 2 ? ~0u : left == 1 ? 0x00ff00ffu : 0u;
#pragma unroll
        for (int n = 0; n < FOURS; ++n) {
            const auto two = __builtin_amdgcn_permlane32_swap(uint32_t(four[n][w]), uint32_t(four[n][w + 1]), false, false);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto both = __builtin_amdgcn_permlane16_swap(two[h], two[h], false, false);
                sc[2 * n + h] = __builtin_amdgcn_perm(both[1], both[0], halves) & keep;
            }
        }
    };
    auto multiply = [&](auto tc, auto hc) __attribute__((always_inline)) {
        constexpr int t = decltype(tc)::value, first = decltype(hc)::value * T::CB / 2;
        static_for<0, T::CB / 2 * T::RB>([&](auto mc) __attribute__((always_inline)) {
            constexpr int i = decltype(mc)::value % T::RB, j = first + decltype(mc)::value / T::RB, b = T::RB + j;
            acc[i][j] = mx4_mfma<t + 2 * (i % 2), t + 2 * (b % 2)>(fa[t][i], fb[t][j], acc[i][j], int(sc[i / 2]), int(sc[b / 2]));
        });
    };

    // what is left of a resource k bytes on (saturated sizes lose k bytes that no tile reaches: see kMaxLd)
    // (in signed integers: a saturating difference of unsigned ones has no scalar form)
    const auto rest = [](uint32_t size, int k) { return uint32_t(max(int(size) - k, 0)); };
    int load_entry = 0;                              // the ring's entry that scales go to next
    auto issue_scales = [&](int panel) __attribute__((always_inline)) {
        char *to = ring + load_entry * T::SBYTES;
        load_entry = load_entry + 1 == T::SRING ? 0 : load_entry + 1;
        const uint32_t past = 8 * panel >= blocks ? kOob : 0u;
#pragma unroll
        for (int i = 0; i < T::SCH; ++i) {
            const int8_t *const at = St[i] + int64_t(panel >> 1) * s_step[i];
            load16_lds(at, bytes_range(at, s_end[i]), s_off[i] | past, to + (i * T::NT + wave * 64) * 16);
        }
    };
    auto issue = [&](int panel, char *st) __attribute__((always_inline)) {
        const int k = panel * T::BK;
        // in the split's last panel, and past it, chunks past its end read as zero
        const uint32_t past = k + q * 16 >= kn ? kOob : 0u;
#pragma unroll
        for (int i = 0; i < T::ACH; ++i)
            load16_lds(At + k, rest(a_size, k), (a_off | past) + uint32_t(i * (T::NT / T::CPR) * p.lda),
                       st + (i * T::NT + wave * 64) * 16);
#pragma unroll
        for (int i = 0; i < T::BCH; ++i)
            load16_lds(Bt + k, rest(b_size, k),
                       (b_off | past) + uint32_t(mx4_b_row<T>(i * (T::NT / T::CPR)) * p.ldb),
                       st + T::A_BYTES + (i * T::NT + wave * 64) * 16);
    };
    // A step goes in halves of B's columns. In the first the second's columns are read, in the second the
    // next step's A and first columns: no more than one step's operands and a half are held. In the
    // middle of a panel's last step the reads of its stage are over, so the barrier comes there: the
    // wave's loads of the next panel have landed, every wave's have after the barrier, and the stage
    // just read is loaded again. (Loads still under way then: those of NSTG - 2 panels, with the scales
    // of half of them.)
    constexpr int LPP = T::ACH + T::BCH;
    constexpr int UNDER_WAY = (T::NSTG - 2) * LPP + (T::NSTG - 2) / 2 * T::SCH;
    typedef std::integral_constant<int, 0> Zero;
    typedef std::integral_constant<int, 1> One;
    if constexpr (!T::LOOP) load_bias(n0);
#pragma unroll
    for (int i = 0; i < T::NSTG; ++i) {
        if (i % 2 == 0) issue_scales(i);
        issue(i, smem + i * STAGE);
    }
    wait_vmcnt<(T::NSTG - 1) * LPP + (T::NSTG / 2 - 1) * T::SCH>();
    asm volatile("s_barrier" ::: "memory");
    typedef std::integral_constant<bool, false> Even;
    typedef std::integral_constant<bool, true> Odd;
    int entry = 0;                                   // the ring's entry of the pair read last
    read_scales(0);
    take_scales(0, Even{});
    read_a(0, Zero{});
    read_b(0, Zero{}, Zero{});
    int stage = 0;                                   // of the pair
    int behind = 0;                                  // panels between a panel read and that of its tile
    auto run = [&](int panel, auto odd) __attribute__((always_inline)) {
        constexpr bool ODD = decltype(odd)::value;
        const int st = (stage + (ODD ? 1 : 0)) * STAGE;
        if constexpr (ODD) stage = stage + 2 == T::NSTG ? 0 : stage + 2;
        const int next = ODD ? stage * STAGE : st + STAGE;
        // MF MFMAs with R reads behind the first of them and L loads behind the others
        const auto spread = [](auto rc, auto lc) __attribute__((always_inline)) {
            constexpr int R = decltype(rc)::value, L = decltype(lc)::value, MF = T::RB * T::CB / 2;
            constexpr int rm = L > 0 ? (MF + 1) / 2 : R < MF ? R : MF, lm = MF - rm > 0 ? MF - rm : 1;
            static_for<0, MF>([&](auto mc) __attribute__((always_inline)) {
                constexpr int m = decltype(mc)::value, n = m - (MF - lm);
                constexpr int r = m < rm ? (m + 1) * R / rm - m * R / rm : 0;
                constexpr int l = n >= 0 ? (n + 1) * L / lm - n * L / lm : 0;
                __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
                if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(kSchedDsRead, r, 0);
                if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(kSchedVmemRead, l, 0);
            });
        };
        constexpr int HALF = T::CB / 2;
        static_assert(T::CB % 2 == 0 && T::STEPS == 2, "halves of two steps");
        read_b(st, Zero{}, One{});
        multiply(Zero{}, Zero{});
        spread(std::integral_constant<int, HALF>{}, Zero{});
        read_a(st, One{});
        read_b(st, One{}, Zero{});
        multiply(Zero{}, One{});
        spread(std::integral_constant<int, T::RB + HALF>{}, Zero{});
        read_b(st, One{}, One{});
        multiply(One{}, Zero{});
        spread(std::integral_constant<int, HALF>{}, Zero{});
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<UNDER_WAY>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        read_a(next, Zero{});
        read_b(next, Zero{}, Zero{});
        if constexpr (ODD) {
            entry = entry + 1 == T::SRING ? 0 : entry + 1;
            read_scales(entry);
        } else {
            issue_scales(panel + T::NSTG - behind);
        }
        issue(panel + T::NSTG - behind, smem + st);
        multiply(One{}, One{});
        spread(std::integral_constant<int, T::RB + HALF + (ODD ? FOURS : 0)>{},
               std::integral_constant<int, LPP + (ODD ? 0 : T::SCH)>{});
        // (behind a tile's last panel comes the first of the next: its scales are whole or masked alike)
        if constexpr (ODD) take_scales(panel + 1 == panels ? 0 : panel + 1, Even{});
        else take_scales(panel + 1, Odd{});
    };
    if constexpr (!T::LOOP) {
        int panel = 0;
        for (; panel + 1 < panels; panel += 2) {
            run(panel, Even{});
            run(panel + 1, Odd{});
        }
        if (panel < panels) run(panel, Even{});
        wait_vmcnt<0>();   // no load is in flight to LDS when the workgroup ends
        mx4_epilogue<T>(p, acc, bias, m0, n0, split, wm, wn);
    } else {
        // The last NSTG panels of a tile load the first of the next, so that its stores and the start
        // of the next run under each other (the grid has fewer workgroups than tiles only where K
        // has NSTG panels).
        for (;;) {
            const int cm0 = m0, cn0 = n0;
            tile += int(gridDim.x);
            const bool more = p.splits == 1 && tile < tiles;
            int panel = 0;
            for (int part = 0; part < 2; ++part) {
                const int end = part == 0 ? panels - T::NSTG : panels;
                for (; panel < end; panel += 2) {
                    run(panel, Even{});
                    run(panel + 1, Odd{});
                }
                if (part == 0 && more) {
                    aim(tile);
                    behind = panels;
                }
            }
            if (!more) wait_vmcnt<0>();
            load_bias(cn0);
            mx4_epilogue<T>(p, acc, bias, cm0, cn0, split, wm, wn);
            if (!more) break;
            behind = 0;
#pragma unroll
            for (int i = 0; i < T::RB; ++i)
#pragma unroll
                for (int j = 0; j < T::CB; ++j) acc[i][j] = f32x4(0.0f);
        }
    }
}

}  // namespace sgemm
