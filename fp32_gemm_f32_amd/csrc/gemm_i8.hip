// gemm_i8.hip -- the C ABI declared in include/gemm_i8.h: validation (pure host code), the
// quick returns, the plan, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <utility>

#include "gemm_i8.h"
#include "kernel_i8.hpp"
#include "kernel_i8_rows.hpp"
#include "ops_common.hpp"

namespace sgemm {
namespace {

constexpr int kMaxK = 131071;               // K * 128 * 128 < 2^31
constexpr int64_t kMaxLd = 8388608;         // 256 rows stay below 2^31 bytes
constexpr int kWorkspaceAlign = 16;

typedef void (*I8Kernel)(I8Args);

// The tiles, smallest first. In microseconds: `c1` and `c2` are a panel of 128 with one and two
// workgroups on every compute unit, `ends` a workgroup's start and stores, `next` what each further
// tile of a workgroup that goes on adds to its panels (its stores, mostly). They and the
// constants of make_plan were fitted to the times of every tile and split of 577 products drawn over
// M of 17 to 16384 and N, K of 64 to 16384, so that the plan's choice costs least: 1.4 % more than
// the best of each on average, 17 % at most (an earlier fit to 219 of them: 2.1 % on 219 others).
// Eight waves serve a tile better than four where one workgroup has a compute unit (2048^3 with
// 128 x 128: 18.2 and 16.5 us at 2 stages), and 4 stages better than 2 there (13.4); in the form for
// any rows each wave joins its own operands' words, and more waves join more (4096 x 4096 x 4097 with
// 128 x 128 and 2 stages: 103 and 108). Tiles and rings whose going costs 0.2 % in all over the
// drawn products are not here.
struct I8Variant {
    const char *name;
    I8Kernel kernel;
    int bm, bn, threads;
    int at_once;     // workgroups on a compute unit
    int loop;        // panels from which a workgroup goes on to another tile, or 0
    double c1, c2, ends, next;
};

template <int BM, int BN, int WGM, int WGN, int NSTG, bool ANY>
constexpr I8Variant tile(const char *name, double c1, double c2, double ends, double next)
{
    typedef I8Tile<BM, BN, WGM, WGN, 128, NSTG> T;
    return {name, &k_gemm_i8<T, ANY>, BM, BN, T::NT, T::LOOP ? 1 : 2, T::LOOP && !ANY ? NSTG : 0, c1, c2, ends, next};
}

const I8Variant kAligned[] = {
    tile<64, 32, 2, 1, 6, false>("i8_64x32", 0.189, 0.27, 2.31, 0.0),
    tile<64, 64, 2, 2, 4, false>("i8_64x64", 0.200, 0.37, 1.84, 0.0),
    tile<64, 128, 2, 4, 3, false>("i8_64x128_w8", 0.298, 0.52, 2.17, 0.0),
    tile<128, 128, 4, 2, 2, false>("i8_128x128", 0.506, 0.95, 1.19, 0.0),
    tile<128, 128, 4, 2, 4, false>("i8_128x128_s4", 0.408, 0.0, 2.04, 3.76),
    tile<128, 256, 2, 4, 3, false>("i8_128x256", 0.644, 0.0, 2.83, 7.49),
    tile<192, 256, 2, 4, 2, false>("i8_192x256", 0.962, 0.0, 3.46, 8.19),
    tile<256, 256, 4, 2, 2, false>("i8_256x256", 1.125, 0.0, 2.20, 7.80),
};
const I8Variant kAny[] = {
    tile<64, 32, 2, 1, 6, true>("i8_64x32", 0.285, 0.46, 1.80, 0.0),
    tile<64, 64, 2, 2, 4, true>("i8_64x64", 0.368, 0.62, 1.85, 0.0),
    tile<64, 128, 2, 2, 3, true>("i8_64x128", 0.418, 0.75, 2.19, 0.0),
    tile<64, 128, 2, 4, 3, true>("i8_64x128_w8", 0.449, 0.78, 1.86, 0.0),
    tile<128, 128, 4, 2, 4, true>("i8_128x128_s4", 0.631, 0.0, 2.33, 0.0),
    tile<192, 128, 2, 4, 3, true>("i8_192x128", 0.709, 0.0, 2.92, 0.0),
    tile<192, 256, 2, 4, 2, true>("i8_192x256", 1.349, 0.0, 3.69, 0.0),
    tile<256, 256, 4, 2, 2, true>("i8_256x256", 1.544, 0.0, 2.56, 0.0),
};
// Few rows: 16 rows, all of K to a workgroup.
const I8Variant kRowsAligned = {"i8_rows16", &k_gemm_i8_rows<I8Rows<1, 1, 8, 4, true>>, 16, 16, 512, 2, 0, 0.0, 0.0, 0.0, 0.0};
const I8Variant kRowsAny = {"i8_rows16", &k_gemm_i8_rows<I8Rows<1, 2, 8, 2, false>>, 16, 32, 512, 2, 0, 0.0, 0.0, 0.0, 0.0};

struct I8Plan {
    const I8Variant *v;
    bool any;
    int tiles_m, tiles_n, splits, k_chunk;
    bool copy_a, copy_b;
    double cost;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// What the plan has to know of an operand: rows on word boundaries, K whole chunks.
struct I8Layout {
    bool a, b;       // A's and B's rows can be loaded as they are
};
I8Layout layout_of(int K, const void *A, int64_t lda, const void *B, int64_t ldb)
{
    const auto ok = [&](const void *p, int64_t ld) {
        return K % 16 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 4 == 0;
    };
    return {ok(A, lda), ok(B, ldb)};
}

constexpr double kLaunch = 2.5;          // us: a kernel's start and end
constexpr double kStreamPerUs = 6.4e6;   // bytes of operands, from the last-level cache too
constexpr double kMostCopied = 4.0e9;    // bytes of workspace a copy may ask for

// Whether workgroups go on to another tile, one to a compute unit.
bool goes_on(const I8Variant &v, int64_t tiles, int splits, int64_t panels, int cus)
{
    return splits == 1 && v.loop > 0 && panels >= v.loop && tiles > cus;
}
// Microseconds of workgroups of `panels` panels each: whole rounds of them and what is left.
double tile_cost(const I8Variant &v, int64_t groups, int splits, int64_t panels, int cus)
{
    const int64_t full = groups / (cus * v.at_once), rest = groups % (cus * v.at_once);
    const int64_t rounds = full + (rest > 0);
    if (goes_on(v, groups, splits, panels, cus))
        return v.c1 * (double(rounds * panels) + 2.7) + v.ends + double(rounds - 1) * v.next;
    const double whole = v.at_once == 2 ? v.c2 : v.c1;
    const double tail = rest == 0 ? 0.0 : rest <= cus ? v.c1 : v.c2;
    return (double(full) * whole + tail) * (double(panels) + 2.7) + double(rounds) * v.ends;
}

// The cheapest of: every tile, K whole or split; rows as they are, in the slower form for any
// alignment, or copied into place first. That form costs a quarter to a half more (measured at
// 8192 x 8192 x 8193 563 against 442 us for 8192^3, 4096 x 4096 x 4097 76 against 61 for 4096^3, 1023 x
// 1025 x 1027 9.4 against 5.3 for 1024^3); the copy costs a launch and its traffic, and the workspace
// (526 and 81 us for the first two with it: the plan takes it for both, for the second wrongly by 6 %).
// The cost orders choices and is no time: it knows no clock under load (368 for 8192 x 8192 x 8193).
I8Plan make_plan(int M, int N, int K, I8Layout rows, int cus, bool workspace)
{
    I8Plan best{};
    const int64_t panels = ceil_div(K, 128);
    const bool any = !(rows.a && rows.b);
    const double bytes = double(M) * K + double(N) * K;
    const double copied = (rows.a ? 0.0 : double(M) * K) + (rows.b ? 0.0 : double(N) * K);
    // what a copy takes of the workspace: rows of whole chunks, up to 16 bytes for one of K = 1
    const double space = (rows.a ? 0.0 : double(M) * round16(K)) + (rows.b ? 0.0 : double(N) * round16(K));
    const auto offer = [&](const I8Plan &p) {
        if (best.v == nullptr || p.cost < best.cost) best = p;
    };
    const auto splits_of = [&](int want) {
        const int64_t chunk = ceil_div(panels, want) * 128;
        return std::pair<int, int>(int(ceil_div(K, chunk)), int(std::min<int64_t>(chunk, K)));
    };
    const auto join_cost = [&](int splits) {
        return splits == 1 ? 0.0 : 2.3 + double(splits + 1) * M * N * 4 / 1.9e6;
    };
    const int most = workspace ? int(std::min<int64_t>(16, std::max<int64_t>(1, panels / 4))) : 1;
    if (M <= 16) {
        // 8 waves share K in panels of 256 (128 in the form for any rows)
        const I8Variant &v = any ? kRowsAny : kRowsAligned;
        for (int want = 1; want <= most; ++want) {
            const auto [s, chunk] = splits_of(want);
            const int64_t groups = ceil_div(N, v.bn) * s;
            if (s > 1 && groups > most_groups(v.threads)) break;     // splits take one launch
            // a panel of every wave takes this long when little else is in flight
            const double turn = any ? double(ceil_div(chunk, 1024)) * 1.4 : double(ceil_div(chunk, 2048)) * 0.8;
            const double step = double(ceil_div(groups, 2 * cus)) * turn;
            const double cost = kLaunch + 1.0 + std::max(step, bytes / 4.6e6 * (any ? 1.25 : 1.0)) +
                                join_cost(s);
            offer({&v, any, 1, int(ceil_div(N, v.bn)), s, chunk, false, false, cost});
        }
        return best;
    }
    const auto offer_tile = [&](const I8Variant &v, bool in_any_form) {
        const bool copies = any && !in_any_form;
        const int64_t tm = ceil_div(M, v.bm), tn = ceil_div(N, v.bn);
        for (int want = 1; want <= most; ++want) {
            const auto [s, chunk] = splits_of(want);
            if (s > 1 && tm * tn * s > 2 * int64_t(cus)) break;
            const double work = tile_cost(v, tm * tn * s, s, ceil_div(chunk, 128), cus), reads = bytes / kStreamPerUs;
            const double body = std::max(work, reads) + 0.02 * std::min(work, reads);   // reads alone tie
            offer({&v, in_any_form, int(tm), int(tn), s, chunk, copies && !rows.a, copies && !rows.b,
                   kLaunch + body + join_cost(s) + (copies ? 4.6 + 2.0 * copied / 6.8e6 : 0.0)});
        }
    };
    if (!any || (workspace && space <= kMostCopied))
        for (const I8Variant &v : kAligned) offer_tile(v, false);
    if (any)
        for (const I8Variant &v : kAny) offer_tile(v, true);
    return best;
}

// Workspace: the splits' sums, then the copies.
struct I8Space {
    int64_t a, b, bytes;      // offsets of the copies, the whole
};
I8Space space_of(const I8Plan &p, int M, int N, int K)
{
    I8Space s{};
    s.a = p.splits > 1 ? round16(int64_t(p.splits) * M * N * 4) : 0;
    s.b = s.a + (p.copy_a ? int64_t(M) * round16(K) : 0);
    s.bytes = s.b + (p.copy_b ? int64_t(N) * round16(K) : 0);
    return s;
}

bool shape_in_limits(int M, int N, int K, int64_t lda, int64_t ldb)
{
    // 16 x 16 is the smallest tile: its count bounds every grid
    const int64_t tiles = ceil_div(M, 16) * ceil_div(N, 16);
    return K <= kMaxK && lda < kMaxLd && ldb < kMaxLd && tiles < (int64_t(1) << 30);
}

// t / d == mulhi(t, mul) >> shift for t < 2^31 and 2^shift < d <= 2^(shift + 1): mul = 2^(32 + shift) / d
// rounded up is too large by less than 1, which adds less than t / 2^(32 + shift) < 1 / d to t / d.
struct Divisor {
    uint32_t mul;
    int shift;
};
Divisor divisor(uint32_t d)
{
    int shift = 0;
    while ((uint64_t(2) << shift) < d) ++shift;
    return {uint32_t(((uint64_t(1) << (32 + shift)) + d - 1) / d), shift};
}

unsigned element_blocks(int64_t total)
{
    return unsigned(std::min<int64_t>((total + 255) / 256, 16384));
}

// The smallest form whose registers hold a row: lanes of a wave to a row for short ones, the
// workgroup for longer ones. 16 chunks to a thread pay only for FP32 rows (4096 x 16384 75 to 62 us;
// 2000 x 20000 bf16 25 to 36, of half as many rows in flight) and many of them (16 x 16384 4.0 to 4.7).
template <int DT>
int quantize(int M, int K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *scales,
             void *stream)
{
    constexpr int SIZE = DT == SGEMM_DTYPE_F32 ? 4 : 2, W = 16 / SIZE;
    const auto rows_from = [&](int64_t row) { return static_cast<const char *>(X) + row * ldx * SIZE; };
    const auto run = [&](auto kern, int rows_per_group) {
        const int64_t most = most_groups(256) * rows_per_group;
        for (int64_t r = 0; r < M; r += most) {
            const int rows = int(std::min<int64_t>(most, M - r));
            const int st = launch(kern, dim3(unsigned(ceil_div(rows, rows_per_group))), dim3(256), stream, rows, K,
                                  rows_from(r), ldx, Q + r * ldq, ldq, scales + r);
            if (st != SGEMM_OK) return st;
        }
        return int(SGEMM_OK);
    };
    const int64_t chunks = ceil_div(K, W);
    if (chunks <= 8) return run(&k_quantize_rows<DT, 1, 8>, 32);
    if (chunks <= 16) return run(&k_quantize_rows<DT, 1, 16>, 16);
    if (chunks <= 32) return run(&k_quantize_rows<DT, 1, 32>, 8);
    if (chunks <= 64) return run(&k_quantize_rows<DT, 1, 64>, 4);
    if (chunks <= 128) return run(&k_quantize_rows<DT, 2, 64>, 4);
    if (chunks <= 256) return run(&k_quantize_rows<DT, 4, 64>, 4);
    if (chunks <= 512) return run(&k_quantize_rows<DT, 2, 256>, 1);
    if (chunks <= 1024) return run(&k_quantize_rows<DT, 4, 256>, 1);
    if (chunks <= 2048) return run(&k_quantize_rows<DT, 8, 256>, 1);
    if constexpr (DT == SGEMM_DTYPE_F32)
        if (chunks <= 4096 && M >= 512) return run(&k_quantize_rows<DT, 16, 256>, 1);
    const int64_t most = most_groups(1024);
    for (int64_t r = 0; r < M; r += most) {
        const int st = launch(&k_quantize_long_rows<DT>, dim3(unsigned(std::min<int64_t>(most, M - r))), dim3(1024),
                              stream, K, rows_from(r), ldx, Q + r * ldq, ldq, scales + r);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int gemm_i8_quantize_rows(int M, int K, const void *X, int x_dtype, int64_t ldx,
                                     int8_t *Q, int64_t ldq, float *scales, void *stream)
{
    if (M < 0 || K < 0) return SGEMM_EINVAL_DIM;
    if (ldx < std::max(K, 1) || ldq < std::max(K, 1)) return SGEMM_EINVAL_LD;
    if (!known_dtype(x_dtype)) return SGEMM_EINVAL_ARG;
    const Region x = region(X, M, K, ldx, dtype_bytes(x_dtype)), q = region(Q, M, K, ldq, 1),
                 s = region(scales, 1, M, M, 4);
    if (bad_region(x, dtype_bytes(x_dtype)) || bad_region(q, 1) || bad_region(s, 4))
        return SGEMM_EINVAL_PTR;
    if (overlaps(q, x) || overlaps(s, x) || overlaps(s, q)) return SGEMM_EALIAS;
    if (M == 0) return SGEMM_OK;
    if (x_dtype == SGEMM_DTYPE_F32) return quantize<SGEMM_DTYPE_F32>(M, K, X, ldx, Q, ldq, scales, stream);
    if (x_dtype == SGEMM_DTYPE_BF16) return quantize<SGEMM_DTYPE_BF16>(M, K, X, ldx, Q, ldq, scales, stream);
    return quantize<SGEMM_DTYPE_F16>(M, K, X, ldx, Q, ldq, scales, stream);
}

extern "C" size_t gemm_i8_workspace_size(int M, int N, int K, const int8_t *A, int64_t lda,
                                         const int8_t *B, int64_t ldb)
{
    if (M <= 0 || N <= 0 || K <= 0 || lda < K || ldb < K || !shape_in_limits(M, N, K, lda, ldb))
        return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    return size_t(space_of(make_plan(M, N, K, layout_of(K, A, lda, B, ldb), cus, true), M, N, K).bytes);
}

extern "C" int gemm_i8(int M, int N, int K, const int8_t *A, int64_t lda, const float *a_scales,
                       const int8_t *B, int64_t ldb, const float *b_scales, const float *bias,
                       void *C, int c_dtype, int64_t ldc, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0) return SGEMM_EINVAL_DIM;
    if (lda < std::max(K, 1) || ldb < std::max(K, 1) || ldc < std::max(N, 1))
        return SGEMM_EINVAL_LD;
    if (!known_dtype(c_dtype)) return SGEMM_EINVAL_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const Region a = region(A, M, K, lda, 1), b = region(B, N, K, ldb, 1),
                 sa = region(a_scales, 1, K ? M : 0, M, 4),
                 sb = region(b_scales, 1, K ? N : 0, N, 4),
                 bi = region(bias, 1, bias ? N : 0, N, 4),
                 c = region(C, M, N, ldc, dtype_bytes(c_dtype)),
                 w = {workspace, workspace_bytes};
    if (bad_region(a, 1) || bad_region(b, 1) || bad_region(sa, 4) || bad_region(sb, 4) ||
        bad_region(bi, 4) || bad_region(c, dtype_bytes(c_dtype)) ||
        bad_region(w, kWorkspaceAlign))
        return SGEMM_EINVAL_PTR;
    for (const Region &r : {a, b, sa, sb, bi})
        if (overlaps(c, r) || overlaps(w, r)) return SGEMM_EALIAS;
    if (overlaps(c, w)) return SGEMM_EALIAS;
    if (!shape_in_limits(M, N, K, lda, ldb)) return SGEMM_ETOO_LARGE;

    I8Args p{};
    p.A = A; p.B = B; p.sa = a_scales; p.sb = b_scales; p.bias = bias; p.C = C;
    p.lda = lda; p.ldb = ldb; p.ldc = ldc;
    p.M = M; p.N = N; p.K = K; p.c_dtype = c_dtype;
    if (K == 0)
        return launch(&k_gemm_i8_empty, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, p);

    int cus = 0;
    int st = device_cus(&cus);
    if (st != SGEMM_OK) return st;
    const I8Layout rows = layout_of(K, A, lda, B, ldb);
    const I8Plan plan = make_plan(M, N, K, rows, cus, workspace_bytes > 0);
    const I8Space space = space_of(plan, M, N, K);
    if (workspace_bytes > 0 && workspace_bytes < size_t(space.bytes)) return SGEMM_EINVAL_ARG;
    if (plan.copy_a || plan.copy_b) {
        const int64_t ld16 = round16(K);
        const int per = int(std::max<int64_t>(1, 2048 / (ld16 / 16)));
        I8Rows16 a16{}, b16{};
        if (plan.copy_a) a16 = {A, static_cast<int8_t *>(workspace) + space.a, lda, M, per, int(ceil_div(M, per))};
        if (plan.copy_b) b16 = {B, static_cast<int8_t *>(workspace) + space.b, ldb, N, per, int(ceil_div(N, per))};
        st = launch(&k_gemm_i8_align, dim3(unsigned(a16.blocks + b16.blocks)), dim3(256), stream, a16, b16, K);
        if (st != SGEMM_OK) return st;
        if (plan.copy_a) { p.A = a16.dst; p.lda = ld16; }
        if (plan.copy_b) { p.B = b16.dst; p.ldb = ld16; }
        p.K = int(ld16);
    }
    p.partial = static_cast<int *>(workspace);
    p.splits = plan.splits; p.k_chunk = plan.splits > 1 ? plan.k_chunk : p.K;
    const I8Variant &v = *plan.v;
    const bool loops = goes_on(v, int64_t(plan.tiles_m) * plan.tiles_n, plan.splits, ceil_div(K, 128), cus);
    // C in parts that one launch each may take, almost always one: no more workgroups than
    // most_groups, rows and columns that a tile past the last of 2^31 - 1 would carry out of an int
    // (split products are one part: make_plan gives them few tiles)
    const int64_t most = loops ? INT64_MAX : most_groups(v.threads), most_rows = int64_t(1) << 30;
    const int64_t part_m = std::min({int64_t(plan.tiles_m), most, most_rows / v.bm});
    const int64_t part_n = std::min({int64_t(plan.tiles_n), most / part_m, most_rows / v.bn});
    const int csize = dtype_bytes(c_dtype);
    const I8Args whole = p;
    for (int64_t tm = 0; tm < plan.tiles_m; tm += part_m)
        for (int64_t tn = 0; tn < plan.tiles_n; tn += part_n) {
            const int64_t m = tm * v.bm, n = tn * v.bn;
            p.tiles_m = int(std::min(part_m, plan.tiles_m - tm));
            p.tiles_n = int(std::min(part_n, plan.tiles_n - tn));
            p.M = int(std::min<int64_t>(M - m, part_m * v.bm));
            p.N = int(std::min<int64_t>(N - n, part_n * v.bn));
            p.A = whole.A + m * p.lda;
            p.B = whole.B + n * p.ldb;
            p.sa = a_scales + m;
            p.sb = b_scales + n;
            p.bias = bias ? bias + n : nullptr;
            p.C = static_cast<char *>(C) + (m * ldc + n) * csize;
            // (2560 x 13056 x 512 to f32, 256 x 256 tiles: rows on lines of 64 bytes 44.5 to 42.0 us, off
            // them 50.6 to 54.8, as each row of a tile ends in parts of a line)
            p.stream = reinterpret_cast<uintptr_t>(p.C) % 64 == 0 && ldc * csize % 64 == 0;
            const Divisor d = divisor(uint32_t(kGroupM) * uint32_t(p.tiles_n));
            p.group_mul = d.mul; p.group_shift = d.shift;
            int64_t groups = int64_t(p.tiles_m) * p.tiles_n * plan.splits;
            if (loops) groups = std::min<int64_t>(groups, cus);
            st = launch(v.kernel, dim3(unsigned(groups)), dim3(v.threads), stream, p);
            if (st != SGEMM_OK) return st;
        }
    if (plan.splits == 1) return SGEMM_OK;
    return launch(&k_gemm_i8_join, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, p);
}

extern "C" int gemm_i8_plan_describe(int M, int N, int K, int64_t lda, int64_t ldb, int num_cus,
                                     char *buf, int buflen)
{
    if (M <= 0 || N <= 0 || K <= 0) return SGEMM_EINVAL_DIM;
    if (lda < K || ldb < K) return SGEMM_EINVAL_LD;
    if (buf == nullptr || buflen <= 0) return SGEMM_EINVAL_ARG;
    if (!shape_in_limits(M, N, K, lda, ldb)) return SGEMM_ETOO_LARGE;
    int cus = num_cus;
    if (cus <= 0) {
        const int st = device_cus(&cus);
        if (st != SGEMM_OK) return st;
    }
    const I8Plan p = make_plan(M, N, K, layout_of(K, nullptr, lda, nullptr, ldb), cus, true);
    const int n = snprintf(buf, size_t(buflen),
                           "{\"name\": \"%s\", \"form\": \"%s\", \"copies\": [%s, %s], \"BM\": %d, "
                           "\"BN\": %d, \"threads\": %d, \"tiles\": [%d, %d], \"splits\": %d, "
                           "\"k_chunk\": %d, \"cost_us\": %.2f, \"workspace_bytes\": %lld}",
                           p.v->name, p.any ? "any" : "aligned",
                           p.copy_a ? "true" : "false", p.copy_b ? "true" : "false", p.v->bm, p.v->bn,
                           p.v->threads, p.tiles_m, p.tiles_n, p.splits, p.k_chunk, p.cost,
                           static_cast<long long>(space_of(p, M, N, K).bytes));
    return n < buflen ? SGEMM_OK : SGEMM_EINVAL_ARG;
}
