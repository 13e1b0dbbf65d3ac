// gemm_i8.hip -- the C ABI declared in include/gemm_i8.h: validation (pure host code), the
// quick returns, the plan, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>

#include "gemm_i8.h"
#include "kernel_i8.hpp"
#include "ops_common.hpp"

namespace sgemm {
namespace {

constexpr int kMaxK = 131071;               // K * 128 * 128 < 2^31
constexpr int64_t kMaxLd = 8388608;         // 256 rows stay below 2^31 bytes
constexpr int kWorkspaceAlign = 16;

typedef void (*I8Kernel)(I8Args);
struct I8Variant {
    const char *name;
    I8Kernel direct, staged;
    int bm, bn, threads;
};

typedef I8Tile<64, 64, 2, 2, 128, 2, true> Tile64;
typedef I8Tile<64, 64, 2, 2, 128, 2, false> Tile64Staged;

const I8Variant kVariants[] = {
    {"i8_64x64", &k_gemm_i8<Tile64>, &k_gemm_i8<Tile64Staged>, 64, 64, Tile64::NT},
};

struct I8Plan {
    const I8Variant *v;
    int tiles_m, tiles_n, splits, k_chunk;
};

int ceil_div(int64_t a, int64_t b) { return int((a + b - 1) / b); }

I8Plan make_plan(int M, int N, int K, int cus)
{
    I8Plan p{};
    p.v = &kVariants[0];
    p.tiles_m = ceil_div(M, p.v->bm);
    p.tiles_n = ceil_div(N, p.v->bn);
    p.splits = 1;
    p.k_chunk = K;
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    if (tiles * 2 <= cus) {
        const int panels = ceil_div(K, 128);
        const int want = std::min<int64_t>(std::min<int64_t>(cus / tiles, 16), panels / 4);
        if (want > 1) {
            p.k_chunk = ceil_div(panels, want) * 128;
            p.splits = ceil_div(K, p.k_chunk);
        }
    }
    return p;
}

size_t plan_bytes(const I8Plan &p, int M, int N)
{
    return p.splits > 1 ? size_t(p.splits) * M * N * 4 : 0;
}

bool shape_in_limits(int M, int N, int K, int64_t lda, int64_t ldb)
{
    // the smallest tile is 64 wide: its tile count bounds every grid
    const int64_t tiles = int64_t(ceil_div(M, 64)) * ceil_div(N, 64);
    return K <= kMaxK && lda < kMaxLd && ldb < kMaxLd && tiles < (int64_t(1) << 26);
}

unsigned element_blocks(int64_t total)
{
    return unsigned(std::min<int64_t>((total + 255) / 256, 16384));
}

// The smallest form whose registers hold a row: a wave to a row for short ones, the
// workgroup for longer ones.
template <int DT>
int quantize(int M, int K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *scales,
             void *stream)
{
    constexpr int W = 16 / (DT == SGEMM_DTYPE_F32 ? 4 : 2);
    const auto run = [&](auto kern, int rows_per_group) {
        return launch(kern, dim3(unsigned(ceil_div(M, rows_per_group))), dim3(256), stream, M, K, X,
                      ldx, Q, ldq, scales);
    };
    if (K <= 64 * W) return run(&k_quantize_rows<DT, 1, 1>, 4);
    if (K <= 256 * W) return run(&k_quantize_rows<DT, 4, 1>, 4);
    if (K <= 512 * W) return run(&k_quantize_rows<DT, 2, 4>, 1);
    if (K <= 1024 * W) return run(&k_quantize_rows<DT, 4, 4>, 1);
    if (K <= 2048 * W) return run(&k_quantize_rows<DT, 8, 4>, 1);
    return launch(&k_quantize_long_rows<DT>, dim3(unsigned(M)), dim3(1024), stream, K, X, ldx, Q,
                  ldq, scales);
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

extern "C" size_t gemm_i8_workspace_size(int M, int N, int K)
{
    if (M <= 0 || N <= 0 || K <= 0 || !shape_in_limits(M, N, K, 1, 1)) return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    return plan_bytes(make_plan(M, N, K, cus), M, N);
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
    I8Plan plan = make_plan(M, N, K, cus);
    const size_t need = plan_bytes(plan, M, N);
    if (need > 0) {
        if (workspace_bytes == 0) {
            plan.splits = 1;
            plan.k_chunk = K;
        } else if (workspace_bytes < need) {
            return SGEMM_EINVAL_ARG;
        }
    }
    p.partial = static_cast<int *>(workspace);
    p.tiles_m = plan.tiles_m; p.tiles_n = plan.tiles_n;
    p.splits = plan.splits; p.k_chunk = plan.k_chunk;
    const bool direct = K % 16 == 0 && lda % 4 == 0 && ldb % 4 == 0 &&
                        reinterpret_cast<uintptr_t>(A) % 4 == 0 &&
                        reinterpret_cast<uintptr_t>(B) % 4 == 0;
    st = launch(direct ? plan.v->direct : plan.v->staged,
                dim3(unsigned(plan.tiles_m * plan.tiles_n * plan.splits)),
                dim3(plan.v->threads), stream, p);
    if (st != SGEMM_OK || plan.splits == 1) return st;
    return launch(&k_gemm_i8_join, dim3(element_blocks(int64_t(M) * N)), dim3(256), stream, p);
}

extern "C" int gemm_i8_plan_describe(int M, int N, int K, int num_cus, char *buf, int buflen)
{
    if (M <= 0 || N <= 0 || K <= 0) return SGEMM_EINVAL_DIM;
    if (buf == nullptr || buflen <= 0) return SGEMM_EINVAL_ARG;
    if (!shape_in_limits(M, N, K, K, K)) return SGEMM_ETOO_LARGE;
    int cus = num_cus;
    if (cus <= 0) {
        const int st = device_cus(&cus);
        if (st != SGEMM_OK) return st;
    }
    const I8Plan p = make_plan(M, N, K, cus);
    const int n = snprintf(buf, size_t(buflen),
                           "{\"name\": \"%s\", \"BM\": %d, \"BN\": %d, \"threads\": %d, "
                           "\"tiles\": [%d, %d], \"splits\": %d, \"k_chunk\": %d, "
                           "\"workspace_bytes\": %zu}",
                           p.v->name, p.v->bm, p.v->bn, p.v->threads, p.tiles_m, p.tiles_n,
                           p.splits, p.k_chunk, plan_bytes(p, M, N));
    return n < buflen ? SGEMM_OK : SGEMM_EINVAL_ARG;
}
