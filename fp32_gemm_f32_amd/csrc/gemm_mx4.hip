// gemm_mx4.hip -- the C ABI declared in include/gemm_mx4.h: validation (pure host code), the quick
// returns, the plan, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <utility>

#include "gemm_mx4.h"
#include "kernel_mx4.hpp"
#include "kernel_mx4_rows.hpp"
#include "kernel_mx4_tiles.hpp"
#include "ops_common.hpp"

namespace sgemm {
namespace {

constexpr int64_t kMaxLd = 8388608;         // 256 rows stay below 2^31 bytes
constexpr int kMaxRows = 1 << 27;           // 16 bytes of each stay below 2^31
constexpr int kWaves = 8;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

unsigned element_blocks(int64_t total) { return unsigned(std::min<int64_t>((total + 255) / 256, 16384)); }

// Rows in parts whose units one launch holds (and a division takes); `each` units to a thread.
typedef void (*Mx4RowKernel)(Mx4RowArgs);
int by_rows(Mx4RowKernel kern, int each, int M, int K, const void *X, int size, int64_t ldx, const uint8_t *Q,
            int64_t ldq, const uint8_t *scales, int64_t lds, void *stream)
{
    Mx4RowArgs p{};
    p.ldx = ldx; p.ldq = ldq; p.lds = lds; p.K = K;
    p.units = int(4 * ceil_div(K, 32));
    p.by_units = divisor(uint32_t(p.units));
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 31) - 256 * each) / p.units);
    for (int64_t r = 0; r < M; r += most) {
        p.M = int(std::min<int64_t>(most, M - r));
        p.X = static_cast<const char *>(X) + r * ldx * size;
        p.Q = const_cast<uint8_t *>(Q) + r * ldq;
        p.scales = const_cast<uint8_t *>(scales) + r * lds;
        const int64_t groups = ceil_div(int64_t(p.M) * p.units, 256 * each);
        const int st = launch(kern, dim3(unsigned(groups)), dim3(256), stream, p);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

typedef void (*Mx4Kernel)(Mx4Args);

// The tiles, smallest first. In microseconds: `c1` and `c2` are a panel of 256 elements with one and two
// workgroups on every compute unit, `ends` a workgroup's start and stores, `next` what each further
// tile of a workgroup that goes on adds to its panels, `less` what a panel takes less with arranged
// scales. They and the constants of make_plan were fitted to the times of every tile and split
// of 870 products drawn over M of 17 to 12000 and N, K of 64 to 16384 (and N of 32001 and 50001): the plan's
// choice costs 1.1 % more than the best of each on average (1.1 % on those left out of the fit). Tiles of
// 128 x 256 and 192 x 256 and a ring of four panels of 128 x 128 would save less than 0.2 % and are not here.
struct Mx4Variant {
    const char *name;
    Mx4Kernel kernel;
    int bm, bn, threads;
    int at_once;     // workgroups on a compute unit
    int loop;        // panels from which a workgroup goes on to another tile, or 0
    double c1, c2, ends, next, less;
};
template <int BM, int BN, int WGM, int WGN, int NSTG>
constexpr Mx4Variant tile(const char *name, double c1, double c2, double ends, double next, double less)
{
    typedef Mx4Tile<BM, BN, WGM, WGN, NSTG> T;
    return {name, &k_mx4_tiles<T>, BM, BN, T::NT, T::LOOP ? 1 : 2, T::LOOP ? NSTG : 0, c1, c2, ends, next, less};
}
const Mx4Variant kTiles[] = {
    tile<64, 32, 2, 1, 6>("mx4_64x32", 0.258, 0.34, 1.12, 0.0, 0.0),
    tile<64, 64, 2, 2, 4>("mx4_64x64", 0.263, 0.43, 1.65, 0.0, 0.0),
    tile<64, 128, 2, 4, 2>("mx4_64x128", 0.501, 0.73, 0.16, 0.0, 0.0),
    tile<128, 128, 4, 2, 2>("mx4_128x128", 0.645, 0.90, 0.0, 0.0, 0.05),
    tile<256, 256, 4, 2, 2>("mx4_256x256", 1.626, 0.0, 3.14, 3.75, 0.08),
};
// Few rows: 16 rows and columns, turns of 512 elements to a wave.
const Mx4Variant kRows = {"mx4_rows16", &k_mx4_rows<kWaves>, 16, 16, 64 * kWaves, 2, 0, 0.0, 0.0, 0.0, 0.0, 0.0};
// For more columns than run at once and a K of a turn to a wave: two and one to a compute unit, which go on.
const Mx4Variant kRowsOn[] = {
    {"mx4_rows16_on8", &k_mx4_rows_on<8>, 16, 16, 512, 2, 1, 0.0, 0.0, 0.0, 0.0, 0.0},
    {"mx4_rows16_on16", &k_mx4_rows_on<16>, 16, 16, 1024, 1, 1, 0.0, 0.0, 0.0, 0.0, 0.0},
};

// The operands, and which of them the tiles can load as they lie: rows on word boundaries, A's of
// whole chunks.
struct Mx4Operands {
    const uint8_t *p[4];      // A, B, and their scales
    int64_t ld[4];
    bool ready(int i, int K) const
    {
        return ld[i] % 4 == 0 && reinterpret_cast<uintptr_t>(p[i]) % 4 == 0 && (i > 0 || K % 32 == 0);
    }
};

struct Mx4Plan {
    const Mx4Variant *v;
    int tiles_m, tiles_n, splits, chunk;
    bool copy[4];             // A, B: into whole chunks; scales: arranged
    double cost;
};

constexpr double kLaunch = 2.5;          // us: a kernel's start and end
constexpr double kFill = 6.7;            // panels that a workgroup's first one takes

// Whether workgroups go on to another tile, as many as run at once.
bool goes_on(const Mx4Variant &v, int64_t tiles, int splits, int64_t panels, int cus)
{
    return splits == 1 && v.loop > 0 && panels >= v.loop && tiles > cus * v.at_once;
}
// Microseconds of workgroups of `panels` panels each: whole rounds of them and what is left.
double tile_cost(const Mx4Variant &v, int64_t groups, int splits, int64_t panels, int cus, bool arranged)
{
    const int64_t full = groups / (cus * v.at_once), rest = groups % (cus * v.at_once);
    const int64_t rounds = full + (rest > 0);
    const double less = arranged ? v.less : 0.0, c1 = v.c1 - less;
    if (goes_on(v, groups, splits, panels, cus))
        return c1 * (double(rounds * panels) + kFill) + v.ends + double(rounds - 1) * v.next;
    const double whole = v.at_once == 2 ? v.c2 - less : c1;
    const double tail = rest == 0 ? 0.0 : rest <= cus ? c1 : v.c2 - less;
    return (double(full) * whole + tail) * (double(panels) + kFill) + double(rounds) * v.ends;
}

// The cheapest of every tile, K whole or split. (The cost orders choices and is no time.)
Mx4Plan make_plan(int M, int N, int K, const Mx4Operands &x, int cus)
{
    Mx4Plan best{};
    const int kb = K / 2;
    const double bytes = (double(M) + double(N)) * K * 17 / 32;
    const auto offer = [&](const Mx4Plan &p) {
        if (best.v == nullptr || p.cost < best.cost) best = p;
    };
    const auto splits_of = [&](int want) {
        const int64_t chunk = ceil_div(ceil_div(kb, 256), want) * 256;
        return std::pair<int, int>(int(ceil_div(kb, chunk)), int(std::min<int64_t>(chunk, kb)));
    };
    const auto join_cost = [&](int splits) {
        return splits == 1 ? 0.0 : 2.0 + double(splits + 1) * M * N * 4 / 1.9e6;
    };
    const int most = int(std::min<int64_t>(16, std::max<int64_t>(1, kb / 512)));
    if (M <= 16) {
        // (8 x 32001 x 2048 11.6 us with a workgroup to 16 columns, 8.7 going on; 1 x 16384 x 4096 9.0 and 9.6)
        const int64_t groups = ceil_div(N, 16), turns = ceil_div(kb, kMx4Turn);
        if (groups > 6 * cus && turns <= 16)
            return {&kRowsOn[turns <= 8 ? 0 : 1], 1, int(groups), 1, kb, {}, kLaunch + bytes / 4.6e6};
        for (int want = 1; want <= most; ++want) {
            const auto [s, chunk] = splits_of(want);
            const int64_t groups = ceil_div(N, kRows.bn) * s;
            if (s > 1 && groups > most_groups(kRows.threads)) break;     // splits take one launch
            const double turn = double(ceil_div(chunk, kMx4Turn * kWaves)) * 0.8;
            const double step = double(ceil_div(groups, 2 * cus)) * turn;
            offer({&kRows, 1, int(ceil_div(N, kRows.bn)), s, chunk, {},
                   kLaunch + 1.0 + std::max(step, bytes / 4.6e6) + join_cost(s)});
        }
        return best;
    }
    // operands off a word's boundary are copied, scales off it arranged; others are where it pays
    const auto traffic = [&](int i) { return 2.0 * double(i % 2 == 0 ? M : N) * K / (i < 2 ? 2 : 32) / 5.0e6; };
    const bool copy_a = !x.ready(0, K), copy_b = !x.ready(1, K), odd_sa = !x.ready(2, K), odd_sb = !x.ready(3, K);
    const double copies = (copy_a ? traffic(0) : 0.0) + (copy_b ? traffic(1) : 0.0);
    for (const Mx4Variant &v : kTiles) {
        const int64_t tm = ceil_div(M, v.bm), tn = ceil_div(N, v.bn);
        for (int want = 1; want <= most; ++want) {
            const auto [s, chunk] = splits_of(want);
            if (s > 1 && tm * tn * s > 2 * int64_t(cus)) break;
            for (const bool arrange : {false, true}) {
                if (arrange && v.less == 0.0 && !odd_sa && !odd_sb) continue;
                const bool sa = odd_sa || arrange, sb = odd_sb || arrange;
                const double moves = (sa || sb || copies > 0.0 ? 3.0 : 0.0) + (sa ? traffic(2) : 0.0) + (sb ? traffic(3) : 0.0);
                offer({&v, int(tm), int(tn), s, chunk, {copy_a, copy_b, sa, sb},
                       kLaunch + tile_cost(v, tm * tn * s, s, ceil_div(chunk, 128), cus, sa && sb) + join_cost(s) + copies + moves});
            }
        }
    }
    return best;
}

// Rows to a workgroup that copies them: about 512 chunks, two to a thread (1023 and 1025 rows of 515 bytes:
// 6.0 us with 2048), more where there are many.
int rows_to_copy(int rows, int64_t ld16)
{
    const int64_t chunks = std::clamp<int64_t>(rows * (ld16 / 16) / 2048, 512, 2048);
    return int(std::max<int64_t>(1, chunks / (ld16 / 16)));
}

// Workgroups of the plan's launch.
int64_t groups_of(const Mx4Plan &p, int kb, int cus)
{
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    return goes_on(*p.v, tiles, p.splits, ceil_div(kb, 128), cus) ? int64_t(cus) * p.v->at_once : tiles * p.splits;
}

// Workspace: the splits' sums, then the copies.
struct Mx4Space {
    int64_t at[4], bytes;     // offsets of the copies, the whole
};
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
Mx4Space space_of(const Mx4Plan &p, int M, int N, int K)
{
    Mx4Space s{};
    s.bytes = p.splits > 1 ? round16(int64_t(p.splits) * M * N * 4) : 0;
    for (int i = 0; i < 4; ++i) {
        s.at[i] = s.bytes;
        if (p.copy[i]) s.bytes += int64_t(i % 2 == 0 ? M : N) * round16(ceil_div(K, i < 2 ? 2 : 32));   // (whole groups of scales, too)
    }
    return s;
}

bool shape_in_limits(int M, int N, int64_t lda, int64_t lda_scales, int64_t ldb, int64_t ldb_scales)
{
    return lda < kMaxLd && ldb < kMaxLd && lda_scales < kMaxLd && ldb_scales < kMaxLd &&
           M < kMaxRows && N < kMaxRows && ceil_div(M, 16) * ceil_div(N, 16) < (int64_t(1) << 30);
}

// Validation of the quantiser and its inverse; `writes` the packed rows and scales, or the values.
int check_rows(int M, int K, const void *X, int dtype, int64_t ldx, const uint8_t *Q, int64_t ldq,
               const uint8_t *scales, int64_t lds, bool writes_codes)
{
    if (M < 0 || K < 0) return SGEMM_EINVAL_DIM;
    const int kb = K / 2 + K % 2, blocks = int(ceil_div(K, 32));
    if (ldx < std::max(K, 1) || ldq < std::max(kb, 1) || lds < std::max(blocks, 1)) return SGEMM_EINVAL_LD;
    if (!known_dtype(dtype)) return SGEMM_EINVAL_ARG;
    const int size = dtype_bytes(dtype);
    const Region x = region(X, M, K, ldx, size), q = region(Q, M, kb, ldq, 1), s = region(scales, M, blocks, lds, 1);
    if (bad_region(x, size) || bad_region(q, 1) || bad_region(s, 1)) return SGEMM_EINVAL_PTR;
    if (overlaps(q, x) || overlaps(s, x) || (writes_codes && overlaps(s, q))) return SGEMM_EALIAS;
    return SGEMM_OK;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int gemm_mx4_quantize(int M, int K, const void *X, int x_dtype, int64_t ldx, uint8_t *Q, int64_t ldq,
                                 uint8_t *scales, int64_t lds, void *stream)
{
    const int st = check_rows(M, K, X, x_dtype, ldx, Q, ldq, scales, lds, true);
    if (st != SGEMM_OK) return st;
    if (M == 0 || K == 0) return SGEMM_OK;
    const int size = dtype_bytes(x_dtype);
    // several units to a thread where there are plenty (8192 x 8192 bf16)
    const bool many = int64_t(M) * ceil_div(K, 32) >= (1 << 18);
    const Mx4RowKernel kern =
        x_dtype == SGEMM_DTYPE_F32    ? (many ? &k_mx4_quantize<SGEMM_DTYPE_F32, 4> : &k_mx4_quantize<SGEMM_DTYPE_F32, 1>)
        : x_dtype == SGEMM_DTYPE_BF16 ? (many ? &k_mx4_quantize<SGEMM_DTYPE_BF16, 4> : &k_mx4_quantize<SGEMM_DTYPE_BF16, 1>)
                                      : (many ? &k_mx4_quantize<SGEMM_DTYPE_F16, 4> : &k_mx4_quantize<SGEMM_DTYPE_F16, 1>);
    return by_rows(kern, many ? 4 : 1, M, K, X, size, ldx, Q, ldq, scales, lds, stream);
}

extern "C" int gemm_mx4_dequantize(int M, int K, const uint8_t *Q, int64_t ldq, const uint8_t *scales, int64_t lds,
                                   void *Y, int y_dtype, int64_t ldy, void *stream)
{
    const int st = check_rows(M, K, Y, y_dtype, ldy, Q, ldq, scales, lds, false);
    if (st != SGEMM_OK) return st;
    if (M == 0 || K == 0) return SGEMM_OK;
    const int size = dtype_bytes(y_dtype);
    const Mx4RowKernel kern = y_dtype == SGEMM_DTYPE_F32    ? &k_mx4_dequantize<SGEMM_DTYPE_F32>
                              : y_dtype == SGEMM_DTYPE_BF16 ? &k_mx4_dequantize<SGEMM_DTYPE_BF16>
                                                            : &k_mx4_dequantize<SGEMM_DTYPE_F16>;
    return by_rows(kern, 1, M, K, Y, size, ldy, Q, ldq, scales, lds, stream);
}

extern "C" size_t gemm_mx4_workspace_size(int M, int N, int K, const uint8_t *A, int64_t lda, const uint8_t *a_scales,
                                          int64_t lda_scales, const uint8_t *B, int64_t ldb,
                                          const uint8_t *b_scales, int64_t ldb_scales)
{
    const int kb = K / 2, blocks = int(ceil_div(K, 32));
    if (M <= 0 || N <= 0 || K <= 0 || K % 2 || lda < kb || ldb < kb || lda_scales < blocks || ldb_scales < blocks ||
        !shape_in_limits(M, N, lda, lda_scales, ldb, ldb_scales))
        return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    const Mx4Operands x = {{A, B, a_scales, b_scales}, {lda, ldb, lda_scales, ldb_scales}};
    return size_t(space_of(make_plan(M, N, K, x, cus), M, N, K).bytes);
}

extern "C" int gemm_mx4(int M, int N, int K, const uint8_t *A, int64_t lda, const uint8_t *a_scales,
                        int64_t lda_scales, const uint8_t *B, int64_t ldb, const uint8_t *b_scales,
                        int64_t ldb_scales, const float *bias, void *C, int c_dtype, int64_t ldc, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0 || K % 2) return SGEMM_EINVAL_DIM;
    const int kb = K / 2, blocks = int(ceil_div(K, 32));
    if (lda < std::max(kb, 1) || ldb < std::max(kb, 1) || lda_scales < std::max(blocks, 1) ||
        ldb_scales < std::max(blocks, 1) || ldc < std::max(N, 1))
        return SGEMM_EINVAL_LD;
    if (!known_dtype(c_dtype)) return SGEMM_EINVAL_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const Region a = region(A, M, kb, lda, 1), b = region(B, N, kb, ldb, 1),
                 sa = region(a_scales, M, blocks, lda_scales, 1), sb = region(b_scales, N, blocks, ldb_scales, 1),
                 bi = region(bias, 1, bias ? N : 0, N, 4), c = region(C, M, N, ldc, dtype_bytes(c_dtype)),
                 w = {workspace, workspace_bytes};
    if (bad_region(a, 1) || bad_region(b, 1) || bad_region(sa, 1) || bad_region(sb, 1) || bad_region(bi, 4) ||
        bad_region(c, dtype_bytes(c_dtype)) || bad_region(w, 16))
        return SGEMM_EINVAL_PTR;
    for (const Region &r : {a, b, sa, sb, bi})
        if (overlaps(c, r) || overlaps(w, r)) return SGEMM_EALIAS;
    if (overlaps(c, w)) return SGEMM_EALIAS;
    if (!shape_in_limits(M, N, lda, lda_scales, ldb, ldb_scales)) return SGEMM_ETOO_LARGE;

    Mx4Args p{};
    p.A = A; p.B = B; p.sa = a_scales; p.sb = b_scales; p.bias = bias; p.C = C;
    p.lda = lda; p.ldb = ldb; p.ldsa = lda_scales; p.ldsb = ldb_scales; p.ldc = ldc;
    p.M = M; p.N = N; p.KB = kb; p.c_dtype = c_dtype;
    if (K == 0) return launch(&k_mx4_empty, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, p);
    int cus = 0;
    int st = device_cus(&cus);
    if (st != SGEMM_OK) return st;
    Mx4Operands x = {{A, B, a_scales, b_scales}, {lda, ldb, lda_scales, ldb_scales}};
    const Mx4Plan plan = make_plan(M, N, K, x, cus);
    if (groups_of(plan, kb, cus) > most_groups(plan.v->threads)) return SGEMM_ETOO_LARGE;
    const Mx4Space space = space_of(plan, M, N, K);
    if (workspace_bytes < size_t(space.bytes)) return SGEMM_EINVAL_ARG;
    const auto place = [&](int i) { return static_cast<uint8_t *>(workspace) + space.at[i]; };
    int64_t step[2] = {16, 16};                  // scales: of a row's groups, and of all of them
    int64_t size[2] = {(M - 1) * lda_scales + blocks, (N - 1) * ldb_scales + blocks};
    Mx4Place placed{};
    placed.bytes = kb;
    placed.count = blocks;
    int64_t places = 0;
    for (int i = 0; i < 2; ++i) {
        const int count = i == 0 ? M : N;
        if (plan.copy[i]) {
            const int per = rows_to_copy(count, round16(kb));
            placed.rows[i] = {reinterpret_cast<const int8_t *>(x.p[i]), reinterpret_cast<int8_t *>(place(i)), x.ld[i], count,
                              per, int(ceil_div(count, per))};
            places += placed.rows[i].blocks;
            x.p[i] = place(i);
            x.ld[i] = round16(kb);
        }
        if (plan.copy[i + 2]) {
            const int across = int(ceil_div(blocks, 64));
            placed.scales[i] = {x.p[i + 2], place(i + 2), x.ld[i + 2], count, int(ceil_div(count, 64)) * across, across};
            places += placed.scales[i].blocks;
            x.p[i + 2] = place(i + 2);
            x.ld[i + 2] = 16;
            step[i] = int64_t(count) * 16;
            size[i] = step[i] * ceil_div(blocks, 16);
        }
    }
    if (places > 0) {
        st = launch(&k_mx4_place, dim3(unsigned(places)), dim3(256), stream, placed);
        if (st != SGEMM_OK) return st;
    }
    p.lda = x.ld[0]; p.ldb = x.ld[1]; p.ldsa = x.ld[2]; p.ldsb = x.ld[3];
    p.sa_step = int(step[0]); p.sb_step = int(step[1]);
    p.partial = static_cast<float *>(workspace);
    p.splits = plan.splits; p.chunk = plan.splits > 1 ? plan.chunk : kb;
    const Mx4Variant &v = *plan.v;
    p.tiles_m = plan.tiles_m; p.tiles_n = plan.tiles_n;
    p.sa_bytes = size[0]; p.sb_bytes = size[1];
    p.A = x.p[0]; p.B = x.p[1]; p.sa = x.p[2]; p.sb = x.p[3];
    // (as the 8-bit product stores C)
    p.stream = reinterpret_cast<uintptr_t>(C) % 64 == 0 && ldc * dtype_bytes(c_dtype) % 64 == 0;
    const Divisor d = divisor(uint32_t(kGroupM) * uint32_t(p.tiles_n));
    p.group_mul = d.mul; p.group_shift = d.shift;
    st = launch(v.kernel, dim3(unsigned(groups_of(plan, kb, cus))), dim3(v.threads), stream, p);
    if (st != SGEMM_OK) return st;
    if (plan.splits == 1) return SGEMM_OK;
    return launch(&k_mx4_join, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, p);
}

extern "C" int gemm_mx4_plan_describe(int M, int N, int K, int num_cus, char *buf, int buflen)
{
    if (M <= 0 || N <= 0 || K <= 0 || K % 2) return SGEMM_EINVAL_DIM;
    if (buf == nullptr || buflen <= 0) return SGEMM_EINVAL_ARG;
    const int kb = K / 2, blocks = int(ceil_div(K, 32));
    if (!shape_in_limits(M, N, kb, blocks, kb, blocks)) return SGEMM_ETOO_LARGE;
    int cus = num_cus;
    if (cus <= 0) {
        const int st = device_cus(&cus);
        if (st != SGEMM_OK) return st;
    }
    const Mx4Plan p = make_plan(M, N, K, {{}, {4, 4, 4, 4}}, cus);
    const int n = snprintf(buf, size_t(buflen),
                           "{\"name\": \"%s\", \"BM\": %d, \"BN\": %d, \"threads\": %d, \"tiles\": [%d, %d], "
                           "\"splits\": %d, \"chunk\": %d, \"cost_us\": %.2f, \"workspace_bytes\": %lld}",
                           p.v->name, p.v->bm, p.v->bn, p.v->threads, p.tiles_m, p.tiles_n, p.splits, 2 * p.chunk, p.cost,
                           static_cast<long long>(space_of(p, M, N, K).bytes));
    return n < buflen ? SGEMM_OK : SGEMM_EINVAL_ARG;
}
