// token_logprobs.hip -- the C ABI declared in include/token_logprobs.h: validation (pure
// host code), how rows are split over workgroups, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernel_logprobs.hpp"
#include "ops_common.hpp"
#include "token_logprobs.h"

namespace sgemm {
namespace {

constexpr int kMaxTop = TOKEN_LOGPROBS_MAX_TOP;
static_assert(kMaxTop == 64, "a wave's list holds one key per lane");

int ceil_div(int64_t a, int64_t b) { return int((a + b - 1) / b); }

struct RowSplit {
    int splits, part_len;
    int64_t part_bytes;
};

// Long rows are split over workgroups where there are fewer rows than compute units, into
// parts of at least kLeastPart elements: one compute unit takes 22 us over a row of 131072 (its
// arithmetic), 32 of them and the join 9.4. Below kLeastRow the join costs what it saves.
constexpr int kLeastPart = 4096, kLeastRow = 65536;
RowSplit split_rows(int M, int V, int top, int cus)
{
    RowSplit r{1, V, 0};
    if (M < cus && V >= kLeastRow) {
        const int want = std::min(ceil_div(2 * cus, M), V / kLeastPart);
        r.part_len = (ceil_div(V, want) + 7) / 8 * 8;
        r.splits = ceil_div(V, r.part_len);
    }
    if (r.splits > 1) r.part_bytes = sizeof(RowPart) + int64_t((top + 1) / 2 * 2) * 8;
    return r;
}
size_t split_bytes(const RowSplit &r, int M)
{
    return r.splits > 1 ? size_t(M) * r.splits * r.part_bytes : 0;
}

typedef void (*RowKernel)(RowArgs);
struct RowLaunch {
    RowKernel kernel;
    int threads;
};
// Logits of half the last-level cache (256 MB) and more are read past it: 2048 x 50000 bf16 (205 MB)
// 38.5 to 36.4 us, 4096 x 131072 188 to 165; 1500 x 50000 (150 MB) 28.0 to 28.3 where it was
// there still and 30.5 to 28.8 where not; 600 x 50001 level.
constexpr int64_t kStreamBytes = int64_t(128) << 20;
bool streamed(int M, int V, int dtype) { return int64_t(M) * V * dtype_bytes(dtype) >= kStreamBytes; }

// Workgroups of more threads for fewer and longer rows, so that enough loads are in flight.
template <int DT, bool TOP> RowLaunch pass_of(int64_t groups, int len, int cus, bool stream)
{
    if (groups <= cus && len >= 32768) return {&k_row_pass<DT, TOP, 1024, 4, false>, 1024};
    if (groups <= 4 * cus && len >= 8192)
        return {stream ? &k_row_pass<DT, TOP, 512, 4, true> : &k_row_pass<DT, TOP, 512, 4, false>, 512};
    return {stream ? &k_row_pass<DT, TOP, 256, 4, true> : &k_row_pass<DT, TOP, 256, 4, false>, 256};
}
template <int DT> RowLaunch pass_kernel(bool top, int64_t groups, int len, int cus, bool stream)
{
    return top ? pass_of<DT, true>(groups, len, cus, stream) : pass_of<DT, false>(groups, len, cus, stream);
}
template <int DT> RowKernel join_kernel(bool top)
{
    return top ? &k_row_join<DT, true> : &k_row_join<DT, false>;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" size_t token_logprobs_workspace_size(int M, int V, int dtype, int top)
{
    if (M <= 0 || V <= 0 || !known_dtype(dtype) || top < 0 || top > kMaxTop || top > V) return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    return split_bytes(split_rows(M, V, top, cus), M);
}

extern "C" int token_logprobs(int M, int V, const void *logits, int dtype, int64_t ld,
                              const void *tokens, int token_bytes, float *logprobs,
                              float *entropy, float *lse, int top, float *top_logprobs,
                              int64_t *top_tokens, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    return token_logprobs_low(M, V, logits, dtype, ld, tokens, token_bytes, logprobs, entropy, lse, nullptr, top,
                              top_logprobs, top_tokens, workspace, workspace_bytes, stream);
}

extern "C" int token_logprobs_low(int M, int V, const void *logits, int dtype, int64_t ld,
                                  const void *tokens, int token_bytes, float *logprobs,
                                  float *entropy, float *lse, float *lse_low, int top,
                                  float *top_logprobs, int64_t *top_tokens, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    if (M < 0 || V < 0 || (M > 0 && V == 0)) return SGEMM_EINVAL_DIM;
    if (ld < std::max(V, 1)) return SGEMM_EINVAL_LD;
    if (!known_dtype(dtype) || (token_bytes != 4 && token_bytes != 8) || top < 0 ||
        top > kMaxTop || (M > 0 && top > V))
        return SGEMM_EINVAL_ARG;
    if (M == 0) return SGEMM_OK;
    const int size = dtype_bytes(dtype);
    const Region x = region(logits, M, V, ld, size), t = region(tokens, 1, M, M, token_bytes),
                 w = {workspace, workspace_bytes};
    const Region out[] = {region(logprobs, 1, M, M, 4),
                          region(entropy, 1, entropy ? M : 0, M, 4),
                          region(lse, 1, lse ? M : 0, M, 4),
                          region(top_logprobs, M, top, top, 4),
                          region(top_tokens, M, top, top, 8),
                          region(lse_low, 1, lse_low ? M : 0, M, 4)};
    if (bad_region(x, size) || bad_region(t, token_bytes) || bad_region(out[0], 4) ||
        bad_region(out[1], 4) || bad_region(out[2], 4) || bad_region(out[3], 4) ||
        bad_region(out[4], 8) || bad_region(out[5], 4) || bad_region(w, 16))
        return SGEMM_EINVAL_PTR;
    for (int i = 0; i < 6; ++i) {
        if (overlaps(out[i], x) || overlaps(out[i], t) || overlaps(out[i], w)) return SGEMM_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return SGEMM_EALIAS;
    }
    if (overlaps(w, x) || overlaps(w, t)) return SGEMM_EALIAS;

    int cus = 0;
    int st = device_cus(&cus);
    if (st != SGEMM_OK) return st;
    RowSplit r = split_rows(M, V, top, cus);
    const size_t need = split_bytes(r, M);
    if (need > 0) {
        if (workspace_bytes == 0) r = RowSplit{1, V, 0};
        else if (workspace_bytes < need) return SGEMM_EINVAL_ARG;
    }
    RowArgs p{};
    p.ld = ld; p.token_bytes = token_bytes;
    p.parts = static_cast<char *>(workspace); p.part_bytes = r.part_bytes;
    p.V = V; p.top = top; p.splits = r.splits; p.part_len = r.part_len;
    const int64_t groups = int64_t(M) * r.splits;
    const bool past_caches = streamed(M, V, dtype);
    RowLaunch pass;
    RowKernel join;
    if (dtype == SGEMM_DTYPE_F32) {
        pass = pass_kernel<SGEMM_DTYPE_F32>(top > 0, groups, r.part_len, cus, past_caches);
        join = join_kernel<SGEMM_DTYPE_F32>(top > 0);
    } else if (dtype == SGEMM_DTYPE_BF16) {
        pass = pass_kernel<SGEMM_DTYPE_BF16>(top > 0, groups, r.part_len, cus, past_caches);
        join = join_kernel<SGEMM_DTYPE_BF16>(top > 0);
    } else {
        pass = pass_kernel<SGEMM_DTYPE_F16>(top > 0, groups, r.part_len, cus, past_caches);
        join = join_kernel<SGEMM_DTYPE_F16>(top > 0);
    }
    // rows that are split are fewer than the compute units: they take one turn
    const int64_t most = most_groups(pass.threads) / r.splits;
    for (int64_t row = 0; row < M; row += most) {
        p.M = int(std::min<int64_t>(most, M - row));
        p.logits = static_cast<const char *>(logits) + row * ld * size;
        p.tokens = static_cast<const char *>(tokens) + row * token_bytes;
        p.logprobs = logprobs + row;
        p.entropy = entropy ? entropy + row : nullptr;
        p.lse = lse ? lse + row : nullptr;
        p.lse_low = lse_low ? lse_low + row : nullptr;
        p.top_logprobs = top_logprobs + row * top;
        p.top_tokens = top_tokens + row * top;
        st = launch(pass.kernel, dim3(unsigned(int64_t(p.M) * r.splits)), dim3(pass.threads), stream, p);
        if (st == SGEMM_OK && r.splits > 1) st = launch(join, dim3(unsigned(p.M)), dim3(256), stream, p);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

extern "C" int token_logprobs_backward(int M, int V, const void *logits, int dtype, int64_t ld,
                                       const void *tokens, int token_bytes, const float *lse,
                                       const float *entropy, const float *g_logprob,
                                       const float *g_entropy, const float *g_lse, void *grad,
                                       int64_t ldg, void *stream)
{
    return token_logprobs_backward_low(M, V, logits, dtype, ld, tokens, token_bytes, lse, nullptr, entropy,
                                       g_logprob, g_entropy, g_lse, grad, ldg, stream);
}

extern "C" int token_logprobs_backward_low(int M, int V, const void *logits, int dtype, int64_t ld,
                                           const void *tokens, int token_bytes, const float *lse,
                                           const float *lse_low, const float *entropy,
                                           const float *g_logprob, const float *g_entropy,
                                           const float *g_lse, void *grad, int64_t ldg,
                                           void *stream)
{
    if (M < 0 || V < 0 || (M > 0 && V == 0)) return SGEMM_EINVAL_DIM;
    if (ld < std::max(V, 1) || ldg < std::max(V, 1)) return SGEMM_EINVAL_LD;
    if (!known_dtype(dtype) || (token_bytes != 4 && token_bytes != 8)) return SGEMM_EINVAL_ARG;
    if (M == 0) return SGEMM_OK;
    const int size = dtype_bytes(dtype);
    const Region x = region(logits, M, V, ld, size), d = region(grad, M, V, ldg, size);
    const Region in[] = {region(tokens, 1, M, M, token_bytes),
                         region(lse, 1, M, M, 4),
                         region(entropy, 1, g_entropy ? M : 0, M, 4),
                         region(g_logprob, 1, g_logprob ? M : 0, M, 4),
                         region(g_entropy, 1, g_entropy ? M : 0, M, 4),
                         region(g_lse, 1, g_lse ? M : 0, M, 4),
                         region(lse_low, 1, lse_low ? M : 0, M, 4)};
    if (bad_region(x, size) || bad_region(d, size)) return SGEMM_EINVAL_PTR;
    for (int i = 0; i < 7; ++i)
        if (bad_region(in[i], i == 0 ? token_bytes : 4)) return SGEMM_EINVAL_PTR;
    const bool in_place = grad == logits && ldg == ld;
    if (!in_place && overlaps(d, x)) return SGEMM_EALIAS;
    for (const Region &r : in)
        if (overlaps(d, r)) return SGEMM_EALIAS;

    GradArgs p{};
    p.token_bytes = token_bytes; p.ld = ld; p.ldg = ldg; p.V = V;
    p.part_len = 16384 / size;
    p.parts = ceil_div(V, p.part_len);
    const bool past_caches = streamed(M, V, dtype);
    auto kern = dtype == SGEMM_DTYPE_F32
                    ? (past_caches ? &k_row_gradient<SGEMM_DTYPE_F32, true> : &k_row_gradient<SGEMM_DTYPE_F32, false>)
                : dtype == SGEMM_DTYPE_BF16
                    ? (past_caches ? &k_row_gradient<SGEMM_DTYPE_BF16, true> : &k_row_gradient<SGEMM_DTYPE_BF16, false>)
                    : (past_caches ? &k_row_gradient<SGEMM_DTYPE_F16, true> : &k_row_gradient<SGEMM_DTYPE_F16, false>);
    const int64_t most = most_groups(kGradThreads) / p.parts;      // 31 rows at least: parts < 2^20
    const auto from = [](const float *v, int64_t row) { return v ? v + row : nullptr; };
    for (int64_t row = 0; row < M; row += most) {
        p.M = int(std::min<int64_t>(most, M - row));
        p.logits = static_cast<const char *>(logits) + row * ld * size;
        p.grad = static_cast<char *>(grad) + row * ldg * size;
        p.tokens = static_cast<const char *>(tokens) + row * token_bytes;
        p.lse = lse + row;
        p.lse_low = from(lse_low, row);
        p.entropy = from(entropy, row);
        p.g_logprob = from(g_logprob, row);
        p.g_entropy = from(g_entropy, row);
        p.g_lse = from(g_lse, row);
        const int st = launch(kern, dim3(unsigned(int64_t(p.M) * p.parts)), dim3(kGradThreads), stream, p);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}
