// gemm_mx4.hip -- the C ABI declared in include/gemm_mx4.h: validation (pure host code), the quick
// returns, the plan, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>

#include "gemm_mx4.h"
#include "kernel_mx4.hpp"
#include "kernel_mx4_rows.hpp"
#include "ops_common.hpp"

namespace sgemm {
namespace {

constexpr int64_t kMaxLd = 8388608;         // 256 rows stay below 2^31 bytes
constexpr int kWaves = 8;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// t / d == mulhi(t, mul) >> shift for t < 2^31 and 2^shift < d <= 2^(shift + 1): mul = 2^(32 + shift) / d
// rounded up is too large by less than 1, which adds less than t / 2^(32 + shift) < 1 / d to t / d.
Mx4Divisor divisor(uint32_t d)
{
    int shift = 0;
    while ((uint64_t(2) << shift) < d) ++shift;
    return {uint32_t(((uint64_t(1) << (32 + shift)) + d - 1) / d), shift};
}

unsigned element_blocks(int64_t total) { return unsigned(std::min<int64_t>((total + 255) / 256, 16384)); }

// Rows in parts whose units one launch holds (and a division takes).
template <typename Kernel, typename Elements>
int by_rows(Kernel kern, int M, int K, Elements *X, int size, int64_t ldx, const uint8_t *Q, int64_t ldq,
            const uint8_t *scales, int64_t lds, void *stream)
{
    Mx4RowArgs p{};
    p.ldx = ldx; p.ldq = ldq; p.lds = lds; p.K = K;
    p.units = int(4 * ceil_div(K, 32));
    p.by_units = divisor(uint32_t(p.units));
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 31) - 256) / p.units);
    for (int64_t r = 0; r < M; r += most) {
        p.M = int(std::min<int64_t>(most, M - r));
        p.X = static_cast<const char *>(static_cast<const void *>(X)) + r * ldx * size;
        p.Q = const_cast<uint8_t *>(Q) + r * ldq;
        p.scales = const_cast<uint8_t *>(scales) + r * lds;
        const int st = launch(kern, dim3(unsigned(ceil_div(int64_t(p.M) * p.units, 256))), dim3(256), stream, p);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

struct Mx4Plan {
    int tiles_m, tiles_n, splits, chunk;
};
Mx4Plan make_plan(int M, int N, int K, int cus)
{
    Mx4Plan p{};
    const int kb = K / 2, turns = int(ceil_div(kb, kMx4Turn));
    p.tiles_m = int(ceil_div(M, 16));
    p.tiles_n = int(ceil_div(N, 16));
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    int want = int(std::min<int64_t>(std::max<int64_t>(1, 2 * cus / tiles), std::max(1, turns / kWaves)));
    want = std::min(want, 16);
    const int64_t chunk = ceil_div(turns, want) * kMx4Turn;
    p.splits = int(ceil_div(kb, chunk));
    p.chunk = int(std::min<int64_t>(chunk, kb));
    return p;
}
size_t space_of(const Mx4Plan &p, int M, int N) { return p.splits > 1 ? size_t(p.splits) * M * N * 4 : 0; }

bool shape_in_limits(int M, int N, int64_t lda, int64_t lda_scales, int64_t ldb, int64_t ldb_scales)
{
    return lda < kMaxLd && ldb < kMaxLd && lda_scales < kMaxLd && ldb_scales < kMaxLd &&
           ceil_div(M, 16) * ceil_div(N, 16) < (int64_t(1) << 30);
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
    auto kern = x_dtype == SGEMM_DTYPE_F32    ? &k_mx4_quantize<SGEMM_DTYPE_F32>
                : x_dtype == SGEMM_DTYPE_BF16 ? &k_mx4_quantize<SGEMM_DTYPE_BF16>
                                              : &k_mx4_quantize<SGEMM_DTYPE_F16>;
    return by_rows(kern, M, K, X, size, ldx, Q, ldq, scales, lds, stream);
}

extern "C" int gemm_mx4_dequantize(int M, int K, const uint8_t *Q, int64_t ldq, const uint8_t *scales, int64_t lds,
                                   void *Y, int y_dtype, int64_t ldy, void *stream)
{
    const int st = check_rows(M, K, Y, y_dtype, ldy, Q, ldq, scales, lds, false);
    if (st != SGEMM_OK) return st;
    if (M == 0 || K == 0) return SGEMM_OK;
    const int size = dtype_bytes(y_dtype);
    auto kern = y_dtype == SGEMM_DTYPE_F32    ? &k_mx4_dequantize<SGEMM_DTYPE_F32>
                : y_dtype == SGEMM_DTYPE_BF16 ? &k_mx4_dequantize<SGEMM_DTYPE_BF16>
                                              : &k_mx4_dequantize<SGEMM_DTYPE_F16>;
    return by_rows(kern, M, K, Y, size, ldy, Q, ldq, scales, lds, stream);
}

extern "C" size_t gemm_mx4_workspace_size(int M, int N, int K, const uint8_t *A, int64_t lda, const uint8_t *a_scales,
                                          int64_t lda_scales, const uint8_t *B, int64_t ldb,
                                          const uint8_t *b_scales, int64_t ldb_scales)
{
    (void)A; (void)B; (void)a_scales; (void)b_scales;
    const int kb = K / 2, blocks = int(ceil_div(K, 32));
    if (M <= 0 || N <= 0 || K <= 0 || K % 2 || lda < kb || ldb < kb || lda_scales < blocks || ldb_scales < blocks ||
        !shape_in_limits(M, N, lda, lda_scales, ldb, ldb_scales))
        return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    return space_of(make_plan(M, N, K, cus), M, N);
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
    const Mx4Plan plan = make_plan(M, N, K, cus);
    if (workspace_bytes < space_of(plan, M, N)) return SGEMM_EINVAL_ARG;
    p.partial = static_cast<float *>(workspace);
    p.splits = plan.splits; p.chunk = plan.chunk;
    // C in parts that one launch each may take, almost always one (split products have few tiles)
    const int64_t most = most_groups(64 * kWaves);
    const int64_t part_m = std::min<int64_t>(plan.tiles_m, most), part_n = std::min<int64_t>(plan.tiles_n, most / part_m);
    const Mx4Args whole = p;
    for (int64_t tm = 0; tm < plan.tiles_m; tm += part_m)
        for (int64_t tn = 0; tn < plan.tiles_n; tn += part_n) {
            const int64_t m = tm * 16, n = tn * 16;
            p.tiles_m = int(std::min(part_m, plan.tiles_m - tm));
            p.tiles_n = int(std::min(part_n, plan.tiles_n - tn));
            p.M = int(std::min<int64_t>(M - m, part_m * 16));
            p.N = int(std::min<int64_t>(N - n, part_n * 16));
            p.A = whole.A + m * lda;
            p.B = whole.B + n * ldb;
            p.sa = whole.sa + m * lda_scales;
            p.sb = whole.sb + n * ldb_scales;
            p.bias = bias ? bias + n : nullptr;
            p.C = static_cast<char *>(C) + (m * ldc + n) * dtype_bytes(c_dtype);
            st = launch(&k_mx4_rows<kWaves>, dim3(unsigned(int64_t(p.tiles_m) * p.tiles_n * plan.splits)),
                        dim3(64 * kWaves), stream, p);
            if (st != SGEMM_OK) return st;
        }
    if (plan.splits == 1) return SGEMM_OK;
    return launch(&k_mx4_join, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, whole);
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
    const Mx4Plan p = make_plan(M, N, K, cus);
    const int n = snprintf(buf, size_t(buflen),
                           "{\"name\": \"mx4_rows16\", \"tiles\": [%d, %d], \"splits\": %d, \"workspace_bytes\": %lld}",
                           p.tiles_m, p.tiles_n, p.splits, static_cast<long long>(space_of(p, M, N)));
    return n < buflen ? SGEMM_OK : SGEMM_EINVAL_ARG;
}
