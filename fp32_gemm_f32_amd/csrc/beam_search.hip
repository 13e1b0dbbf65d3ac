// beam_search.hip -- the C ABI declared in include/beam_search.h: validation (pure host code), how
// rows are split over workgroups, the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "beam_search.h"
#include "kernel_beams.hpp"
#include "ops_common.hpp"

namespace sgemm {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct BeamSplit {
    int splits, part_len;
    int64_t part_bytes;
};

// Long rows are split over workgroups where there are fewer rows than compute units, into parts of
// about kPart elements (4 rows of 131072 f32 into 8, 16 and 24 parts: 11.3, 10.6, 11.0 us with the second
// kernel, which joins the parts either way; 32 rows of 32001 bf16 into 2, 4 and 8: 10.1, 10.0, 9.7; 185
// rows of 50001 f16 into 2, 4 and 8: 14.1, 12.8, 13.9).
constexpr int kPart = 8192;
BeamSplit split_beams(int64_t rows, int V, int top, int cus)
{
    BeamSplit r{1, V, 0};
    if (rows < cus && V >= 2 * kPart) {
        const int want = int(std::min<int64_t>(ceil_div(3 * cus, rows), ceil_div(V, kPart)));
        r.part_len = int((ceil_div(V, want) + 7) / 8 * 8);
        r.splits = int(ceil_div(V, r.part_len));
    }
    r.part_bytes = sizeof(RowPart) + int64_t((top + 1) / 2 * 2) * 8;
    return r;
}
size_t beam_bytes(const BeamSplit &r, int64_t rows) { return size_t(rows * r.splits * r.part_bytes); }

typedef void (*BeamKernel)(BeamArgs);
struct BeamLaunch {
    BeamKernel kernel;
    int threads;
};
// Longer parts take more threads (1024 rows of 131072 bf16 with 512 and 1024: 60.2 and 56.2 us; 512 rows of
// 32001 with 256, 512 and 1024: 16.6, 15.6, 17.2). Logits of half the last-level cache and more are
// read past it (the former with 512 threads in two parts: 57.0 instead of 61.5).
constexpr int64_t kStreamBytes = int64_t(128) << 20;
template <int DT> BeamLaunch beam_pass(int len, bool stream)
{
    if (len >= 65536)
        return {stream ? &k_beam_pass<DT, 1024, 2, true> : &k_beam_pass<DT, 1024, 2, false>, 1024};
    if (len >= 2 * kPart)
        return {stream ? &k_beam_pass<DT, 512, 2, true> : &k_beam_pass<DT, 512, 2, false>, 512};
    return {stream ? &k_beam_pass<DT, 256, 2, true> : &k_beam_pass<DT, 256, 2, false>, 256};
}

// Whether a state's pieces overlap (or lie in each other, in an order that is not looked into).
bool overlapping(int64_t rows, int64_t row, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t run)
{
    struct Dim { int64_t n, step; } d[3] = {{rows, row}, {n1, s1}, {n2, s2}};
    std::sort(d, d + 3, [](const Dim &a, const Dim &b) { return a.step < b.step; });
    __int128 extent = run;
    for (const Dim &x : d) {
        if (x.n <= 1) continue;
        if (x.step < extent) return true;
        extent += static_cast<__int128>(x.n - 1) * x.step;
    }
    return false;
}
// Bytes from a region's first to its last, saturated.
uint64_t extent_of(int64_t rows, int64_t row, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t run)
{
    const __int128 n = static_cast<__int128>(rows - 1) * row + static_cast<__int128>(n1 - 1) * s1 +
                       static_cast<__int128>(n2 - 1) * s2 + run;
    const __int128 most = static_cast<__int128>(1) << 62;
    return uint64_t(n < most ? n : most);
}
// One side of a state.
struct Side {
    const beam_state *state;
    bool written;
    uint64_t from, bytes;
};
// Its bytes by their strides from the largest on (counts of 1 and strides of 0 add none).
struct Span {
    int64_t run;
    bool in_place;
    int levels = 0;
    struct { int64_t n, step; } level[3];

    Span(const Side &x, int64_t rows) : run(x.state->run), in_place(x.state->src == x.state->dst)
    {
        const beam_state &s = *x.state;
        const int64_t n[3] = {rows, s.count1, s.count2};
        const int64_t step[3] = {x.written ? s.dst_row : s.src_row, x.written ? s.dst_step1 : s.src_step1,
                                 x.written ? s.dst_step2 : s.src_step2};
        for (int i = 0; i < 3; ++i) {
            if (n[i] <= 1 || step[i] == 0) continue;
            int at = levels++;
            for (; at > 0 && level[at - 1].step < step[i]; --at) level[at] = level[at - 1];
            level[at] = {n[i], step[i]};
        }
    }
    // from the first byte to the last of the levels from k on, saturated
    uint64_t extent(int k) const
    {
        const __int128 most = static_cast<__int128>(1) << 62;
        __int128 sum = run;
        for (; k < levels; ++k) sum = std::min(most, sum + static_cast<__int128>(level[k].n - 1) * level[k].step);
        return uint64_t(sum);
    }
};
// Whether the levels from k on of b, which starts d bytes behind a, hold none of a's bytes: those that
// end before b starts, and slices of a common stride. Of such a stride's periods, a's parts lie at their
// start and b's r behind it. Where b's do not reach into the next period they meet a's of the same one
// at most, always r behind them; else, where a's end before r, those of the next one, which start s - r
// behind b's. Anything else counts as an overlap, and so do slices of the inner strides but of
// states that are both reordered in place.
bool apart(const Span &a, const Span &b, uint64_t d, int k)
{
    if (d >= a.extent(k)) return true;
    if (k == a.levels || k == b.levels || a.level[k].step != b.level[k].step) return false;
    const uint64_t s = uint64_t(a.level[k].step), r = d % s, of_a = a.extent(k + 1), of_b = b.extent(k + 1);
    if (of_a > s || of_b > s) return false;
    if (r >= of_a && r + of_b <= s) return true;
    if (!a.in_place || !b.in_place) return false;
    if (r + of_b <= s) return apart(a, b, r, k + 1);
    return of_a <= r && apart(b, a, s - r, k + 1);
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" size_t beam_step_workspace_size(int B, int W, int V, int dtype, int top)
{
    if (B <= 0 || W <= 0 || W > BEAM_MAX || V <= 0 || !known_dtype(dtype) || top <= 0 || top > BEAM_MAX) return 0;
    int cus = 0;
    if (device_cus(&cus) != SGEMM_OK) return 0;
    const int64_t rows = int64_t(B) * W;
    return beam_bytes(split_beams(rows, V, top, cus), rows);
}

extern "C" int beam_step(int B, int W, int V, const void *logits, int dtype, int64_t ld, const float *scores,
                         const uint8_t *finished, int64_t pad_token, int top, float *out_scores,
                         int64_t *out_beams, int64_t *out_tokens, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    if (B < 0 || W < 0 || V < 0 || (B > 0 && V == 0)) return SGEMM_EINVAL_DIM;
    if (ld < std::max(V, 1)) return SGEMM_EINVAL_LD;
    if (!known_dtype(dtype) || (B > 0 && (W < 1 || W > BEAM_MAX || top < 1 || top > BEAM_MAX)))
        return SGEMM_EINVAL_ARG;
    if (B == 0) return SGEMM_OK;
    const int size = dtype_bytes(dtype);
    const int64_t rows = int64_t(B) * W;
    const Region x = region(logits, rows, V, ld, size), s = region(scores, 1, rows, rows, 4),
                 f = region(finished, 1, finished ? rows : 0, rows, 1), w = {workspace, workspace_bytes};
    const Region out[] = {region(out_scores, B, top, top, 4), region(out_beams, B, top, top, 8),
                          region(out_tokens, B, top, top, 8)};
    if (bad_region(x, size) || bad_region(s, 4) || bad_region(out[0], 4) || bad_region(out[1], 8) ||
        bad_region(out[2], 8) || bad_region(w, 16))
        return SGEMM_EINVAL_PTR;
    for (int i = 0; i < 3; ++i) {
        for (const Region &r : {x, s, f, w})
            if (overlaps(out[i], r)) return SGEMM_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return SGEMM_EALIAS;
    }
    for (const Region &r : {x, s, f})
        if (overlaps(w, r)) return SGEMM_EALIAS;

    int cus = 0;
    int st = device_cus(&cus);
    if (st != SGEMM_OK) return st;
    const BeamSplit r = split_beams(rows, V, top, cus);
    if (workspace_bytes < beam_bytes(r, rows)) return SGEMM_EINVAL_ARG;
    BeamArgs p{};
    p.ld = ld; p.pad_token = pad_token;
    p.part_bytes = r.part_bytes;
    p.W = W; p.V = V; p.top = top; p.splits = r.splits; p.part_len = r.part_len;
    p.by_top = divisor(uint32_t(top)); p.by_splits = divisor(uint32_t(r.splits));
    const bool past_caches = rows * V * size >= kStreamBytes;
    const BeamLaunch pass =
        dtype == SGEMM_DTYPE_F32    ? beam_pass<SGEMM_DTYPE_F32>(r.part_len, past_caches)
        : dtype == SGEMM_DTYPE_BF16 ? beam_pass<SGEMM_DTYPE_BF16>(r.part_len, past_caches)
                                    : beam_pass<SGEMM_DTYPE_F16>(r.part_len, past_caches);
    // requests to a launch (rows that are split are fewer than the compute units: one turn)
    const int64_t most = most_groups(pass.threads) / r.splits / W;
    for (int64_t b = 0; b < B; b += most) {
        const int64_t n = std::min<int64_t>(most, B - b), row = b * W;
        p.logits = static_cast<const char *>(logits) + row * ld * size;
        p.scores = scores + row;
        p.finished = finished ? finished + row : nullptr;
        p.parts = static_cast<char *>(workspace) + row * r.splits * r.part_bytes;
        p.out_scores = out_scores + b * top;
        p.out_beams = out_beams + b * top;
        p.out_tokens = out_tokens + b * top;
        st = launch(pass.kernel, dim3(unsigned(n * W * r.splits)), dim3(pass.threads), stream, p);
        if (st == SGEMM_OK) st = launch(&k_beam_choice, dim3(unsigned(n)), dim3(kChoiceThreads), stream, p);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

extern "C" int reorder_beams(int B, int W, const void *beams, int beam_bytes, const beam_state *states, int count,
                             void *stream)
{
    if (B < 0 || W < 0 || count < 0) return SGEMM_EINVAL_DIM;
    if (count > 0 && states == nullptr) return SGEMM_EINVAL_PTR;
    const int64_t rows = int64_t(B) * W;
    for (int i = 0; i < count; ++i) {
        const beam_state &s = states[i];
        for (int64_t v : {s.src_row, s.dst_row, s.count1, s.src_step1, s.dst_step1, s.count2, s.src_step2,
                          s.dst_step2, s.run})
            if (v < 0) return SGEMM_EINVAL_DIM;
    }
    for (int i = 0; i < count; ++i) {
        const beam_state &s = states[i];
        if (s.count1 && s.count2 && s.run &&
            overlapping(rows, s.dst_row, s.count1, s.dst_step1, s.count2, s.dst_step2, s.run))
            return SGEMM_EINVAL_LD;
    }
    if ((beam_bytes != 4 && beam_bytes != 8) || (rows > 0 && W > BEAM_MAX)) return SGEMM_EINVAL_ARG;
    if (rows == 0 || count == 0) return SGEMM_OK;
    const Region idx = region(beams, 1, rows, rows, beam_bytes);
    if (bad_region(idx, beam_bytes)) return SGEMM_EINVAL_PTR;
    std::vector<Side> sides;
    try {
        sides.reserve(size_t(count) * 2);
    } catch (...) {
        return SGEMM_ELAUNCH;
    }
    bool large = false;
    for (int i = 0; i < count; ++i) {
        const beam_state &s = states[i];
        if (!s.count1 || !s.count2 || !s.run) continue;
        if (s.src == nullptr || s.dst == nullptr) return SGEMM_EINVAL_PTR;
        const bool same = s.src_row == s.dst_row && (s.count1 == 1 || s.src_step1 == s.dst_step1) &&
                          (s.count2 == 1 || s.src_step2 == s.dst_step2);
        const uint64_t bytes = extent_of(rows, s.dst_row, s.count1, s.dst_step1, s.count2, s.dst_step2, s.run);
        sides.push_back({&s, true, reinterpret_cast<uintptr_t>(s.dst), bytes});
        if (s.src != s.dst)
            sides.push_back({&s, false, reinterpret_cast<uintptr_t>(s.src),
                             extent_of(rows, s.src_row, s.count1, s.src_step1, s.count2, s.src_step2, s.run)});
        else if (!same) return SGEMM_EALIAS;
        const __int128 columns = static_cast<__int128>(s.count1) * s.count2 * ceil_div(s.run, 16);
        large = large || columns >= (int64_t(1) << 31) - kReorderThreads;
        if (overlaps({s.dst, bytes}, idx)) return SGEMM_EALIAS;
    }
    std::sort(sides.begin(), sides.end(), [](const Side &a, const Side &b) { return a.from < b.from; });
    for (size_t i = 0; i < sides.size(); ++i)
        for (size_t j = i + 1; j < sides.size() && sides[j].from - sides[i].from < sides[i].bytes; ++j)
            if ((sides[i].written || sides[j].written) &&
                !apart({sides[i], rows}, {sides[j], rows}, sides[j].from - sides[i].from, 0))
                return SGEMM_EALIAS;
    if (large) return SGEMM_ETOO_LARGE;

    auto kern = W <= 4 ? &k_reorder<4> : W <= 8 ? &k_reorder<8> : W <= 16 ? &k_reorder<16>
              : W <= 32 ? &k_reorder<32> : &k_reorder<64>;
    const int64_t most = most_groups(kReorderThreads);
    ReorderArgs p{};
    p.beam_bytes = beam_bytes; p.W = W;
    int64_t groups = 0;
    const auto flush = [&]() {
        const int st = p.count == 0 ? int(SGEMM_OK)
                                    : launch(kern, dim3(unsigned(groups)), dim3(kReorderThreads), stream, p);
        p.count = 0;
        groups = 0;
        return st;
    };
    // requests outermost where one launch does not hold them: a launch has one table of beams
    int64_t step = B;
    for (int i = 0; i < count; ++i) {
        const beam_state &s = states[i];
        if (!s.count1 || !s.count2 || !s.run) continue;
        step = std::min(step, most / ceil_div(s.count1 * s.count2 * ceil_div(s.run, 16), kReorderThreads));
    }
    for (int64_t b = 0; b < B; b += step) {
        const int64_t n = std::min<int64_t>(step, B - b);
        p.beams = static_cast<const char *>(beams) + b * W * beam_bytes;
        for (int i = 0; i < count; ++i) {
            const beam_state &s = states[i];
            if (!s.count1 || !s.count2 || !s.run) continue;
            StateArgs a{};
            a.src = static_cast<const char *>(s.src) + b * W * s.src_row;
            a.dst = static_cast<char *>(s.dst) + b * W * s.dst_row;
            a.src_row = s.src_row; a.dst_row = s.dst_row;
            a.src_step1 = s.src_step1; a.dst_step1 = s.dst_step1;
            a.src_step2 = s.src_step2; a.dst_step2 = s.dst_step2;
            a.run = s.run;
            a.count2 = int(s.count2);
            a.chunks = int(ceil_div(s.run, 16));
            a.columns = int(s.count1 * s.count2 * a.chunks);
            a.blocks = int(ceil_div(a.columns, kReorderThreads));
            a.by_blocks = divisor(uint32_t(a.blocks));
            a.by_chunks = divisor(uint32_t(a.chunks));
            a.by_count2 = divisor(uint32_t(a.count2));
            if (p.count == kStates || groups + n * a.blocks > most) {
                const int st = flush();
                if (st != SGEMM_OK) return st;
            }
            p.first[p.count] = int(groups);
            p.states[p.count++] = a;
            groups += n * a.blocks;
        }
        const int st = flush();
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}
