// kernel_beams.hpp -- kernels of beam_search.h: one pass over each beam's row of logits for its
// log-sum-exp and likeliest tokens, the choice among a request's beams, and the reordering of
// states.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "beam_search.h"
#include "kernel_logprobs.hpp"
#include "kernel_mfma.hpp"
#include "ops_common.hpp"

namespace sgemm {

struct BeamArgs {
    const void *logits;
    int64_t ld;
    const float *scores;
    const uint8_t *finished;   // or NULL
    int64_t pad_token;
    float *out_scores;
    int64_t *out_beams, *out_tokens;
    char *parts;               // part s of row i at (i * splits + s) * part_bytes
    int64_t part_bytes;
    int W, V, top, splits, part_len;
    Divisor by_top, by_splits;
};

// ------------------------------------------------------------------ a beam's row --------
// Running peak m and s = sum 2^(x L - c), L = log2 e as FP32 has it and c = m L: one multiply-add and one
// exponential to an element. What FP32 rounds off here is either known (c is taken as it was rounded),
// random in sign from term to term, or, as L is off by 1.3e-8 of itself, that much of the row's entropy,
// nearly the same for all of a request's beams. Which of two beams' tokens comes first hangs on such
// differences. beam_rescale rounds both its products, so that a sum goes from one c as it was rounded to
// another: a multiply-add in place of one of them would rescale by 2^(half a step of c) each time, even
// where the peak stays.
// Up to kFar a step of c is 128 at most, so that sums of 2^31 terms stay in range. Beyond, logits that
// differ do so by 128 and more, also from those up to it: a term, there 2^((x - m) L), is 1 or 0, and so
// is the factor between two peaks one of which lies beyond, for which 2^(their difference) will do.
constexpr float kFar = 1073741824.0f;                  // 2^30
constexpr double kNats = 1.0 / double(kLog2e);         // of a base-2 logarithm by L
__device__ inline bool beam_near(float m) { return __builtin_fabsf(m) <= kFar; }
// What a sum over peak `from` is multiplied by to be one over `to`, a larger one or the same.
__device__ inline float beam_rescale(float from, float to)
{
#pragma clang fp contract(off)
    const float near = from * kLog2e - to * kLog2e, far = from - to;
    return __builtin_amdgcn_exp2f(__builtin_fmaxf(-from, to) <= kFar ? near : far);
}
struct BeamStats {
    float m = kLowest, s = 0.0f;

    __device__ void raise(float to)
    {
        const float next = __builtin_fmaxf(m, to);
        s *= beam_rescale(m, next);
        m = next;
    }
    // n elements with m already raised to them
    template <int N> __device__ void add(const float (&x)[N])
    {
        if (!beam_near(m)) {
#pragma unroll
            for (int j = 0; j < N; ++j) s += __builtin_amdgcn_exp2f((x[j] - m) * kLog2e);
        } else {
            const float c = m * kLog2e;
#pragma unroll
            for (int j = 0; j < N; ++j) s += __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], kLog2e, -c));
        }
    }
};

// Every thread gets the workgroup's joined sums, in the same order each time.
template <int NT> __device__ inline BeamStats join_beam_stats(StatsShared<NT> &sh, BeamStats st)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    st.raise(wave_reduce(st.m, [](float a, float b) { return __builtin_fmaxf(a, b); }));
    st.s = wave_reduce(st.s, [](float a, float b) { return a + b; });
    if (lane == 0) { sh.m[wave] = st.m; sh.s[wave] = st.s; }
    __syncthreads();
    BeamStats all;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) all.m = __builtin_fmaxf(all.m, sh.m[w]);
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        BeamStats one;
        one.m = sh.m[w];
        one.s = sh.s[w];
        one.raise(all.m);
        all.s += one.s;
    }
    return all;
}

// One workgroup per (row, part): the part's peak and sum, and its `top` largest logits as keys
// (key_of) in descending order, 0 for those it is too short for. Rows of finished beams are left
// out. A thread's elements: up to one of the head before the first 16-byte boundary, the chunks tid,
// tid + NT, ... of 16 bytes, up to one of the tail. Bound by memory and, nearly as much, by the
// exponentials: 1024 rows of 131072 bf16 take 53.4 us (5.0 TB/s). Registers are kept to 64, so that a compute
// unit holds 32 waves (more loads to a thread, or the next ones ahead of these, cost waves: 60 us).
template <int DT, int NT, int U, bool STREAM>
__global__ __launch_bounds__(NT, 8) void k_beam_pass(BeamArgs p)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    // (in shorter parts it costs more than it saves: 4 rows of 131072 f32 10.9 and 11.3 us)
    constexpr bool APART = NT == 1024;
    __shared__ StatsShared<NT> stats;
    __shared__ TopShared<NT> tops;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / p.splits;
    const int part = blockIdx.x % p.splits;
    if (p.finished && p.finished[row]) return;
    const int first = part * p.part_len;                  // this part's elements of the row
    const int n = min(p.part_len, p.V - first);
    const T *x = static_cast<const T *>(p.logits) + row * p.ld + first;
    const int head = min(n, int((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
    const int chunks = (n - head) / W;
    const int tail = head + chunks * W;                   // first element of the tail
    const T *body = x + head;
    if (tid == 0) { tops.n_cand = 0; tops.n_threads = 0; }

    BeamStats st;
    Pack<T, W> b[U];
    // the best group: its value in key order, and its first element; the second best's value
    uint32_t best = 0, second = 0;
    int best_at = tid < head ? tid : tid < chunks ? head + tid * W : tail + tid;
    const bool empty = best_at >= n;
    auto note = [&](float peak, int at) __attribute__((always_inline)) {
        const uint32_t o = ordered(peak);
        best_at = o > best ? at : best_at;
        if constexpr (APART) second = max(second, min(o, best));
        best = max(best, o);
    };
    float edge[2] = {0.0f, 0.0f};                         // the thread's head and tail elements
    auto take1 = [&](int at, float &v) __attribute__((always_inline)) {
        v = Elem<DT>::widen(x[at]);
        note(v, at);
        st.raise(v);
        const float one[1] = {v};
        st.add(one);
    };
    auto load = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            b[u] = load_chunk_of<STREAM, T, W>(body + int64_t(min(c + u * NT, chunks - 1)) * W);
    };
    auto widen = [&](float *v, int u, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = Elem<DT>::widen(b[u].v[j]);
        float peak = v[0];
#pragma unroll
        for (int j = 1; j < W; ++j) peak = __builtin_fmaxf(peak, v[j]);
        note(peak, head + (c + u * NT) * W);
        return peak;
    };
    if (tid < head) take1(tid, edge[0]);
    int c = tid;
    for (; c + (U - 1) * NT < chunks; c += U * NT) {
        float v[U * W], peak = kNegInf;
        load(c);
#pragma unroll
        for (int u = 0; u < U; ++u) peak = __builtin_fmaxf(peak, widen(v + u * W, u, c));
        st.raise(peak);
        st.add(v);
    }
    if (c < chunks) {                                     // fewer than U are left
        load(c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u * NT >= chunks) break;
            float v[W];
            st.raise(widen(v, u, c));
            st.add(v);
        }
    }
    if (tid < n - tail) take1(tail + tid, edge[1]);

    const BeamStats all = join_beam_stats(stats, st);     // a barrier: n_cand is set
    RowPart *out = reinterpret_cast<RowPart *>(p.parts + int64_t(blockIdx.x) * p.part_bytes);
    if (tid == NT - 1) *out = RowPart{all.m, all.s, 0.0f, 0.0f};
    uint64_t *keys = reinterpret_cast<uint64_t *>(out + 1);
    auto emit = [&](int r, uint64_t k) { keys[r] = k - uint32_t(first); };    // indices in the row
    if (tid < p.top && tid >= n) keys[tid] = 0;
    const int top = min(p.top, n);
    const uint64_t mine = empty ? 0 : uint64_t(best) << 32 | (0xffffffffu - uint32_t(best_at));
    uint64_t floor = top_bound(tops, mine, top);
    // the bound's group reaches W - 1 elements behind its first
    floor = max(floor - min(uint32_t(floor), uint32_t(W - 1)), uint64_t(1));
    // Where b holds all of a thread's chunks they are looked at there. Else the thread is listed, and all
    // threads look at the listed ones' chunks; APART: but where only its best group reaches the bound
    // it loads that alone (16 bytes here and there are a line of 128 each: of 1024 rows of 131072 bf16
    // and 16 of each, 12 % more is read without, 56.7 and 54.3 us).
    if (mine >= floor) {
        if (chunks <= U * NT) {
            static_assert(U * W <= 32, "a bit for each element");
            const int mine_n = tid < chunks ? (chunks - tid + NT - 1) / NT * W : 0;
            add_candidates<DT>(tops, b, mine_n == 32 ? 0xffffffffu : (1u << mine_n) - 1, floor,
                               [&](int i) { return head + (tid + i / W * NT) * W + i % W; });
            if (tid < head) add_candidate(tops, key_of(edge[0], uint32_t(tid)), floor);
            if (tid < n - tail) add_candidate(tops, key_of(edge[1], uint32_t(tail + tid)), floor);
        } else if (!APART || second >= uint32_t(floor >> 32)) {
            tops.threads[atomicAdd(&tops.n_threads, 1)] = tid;
        } else if (best_at < head || best_at >= tail) {
            add_candidate(tops, key_of(edge[best_at < head ? 0 : 1], uint32_t(best_at)), floor);
        } else {
            const Pack<T, W> one[1] = {load_pack<T, W>(x + best_at)};
            add_candidates<DT>(tops, one, (1u << W) - 1, floor, [&](int j) { return best_at + j; });
        }
    }
    __syncthreads();
    int found = tops.n_cand;
    const int listed = tops.n_threads;
    if (found <= kCandidates && listed == 0) {
        rank_top(tops, found, top, emit);
        return;
    }
    __syncthreads();                                      // all have read both before either changes
    if (found > kCandidates) {                            // list them all
        if (tid == 0) { tops.n_cand = 0; tops.n_threads = 0; }
        __syncthreads();
        if (mine >= floor) tops.threads[atomicAdd(&tops.n_threads, 1)] = tid;
        __syncthreads();
        found = 0;
    }
    // the threads' chunks, and one more slot for their head and tail
    const int per = (chunks + NT - 1) / NT + 1;
    auto look = [&](int slot, uint64_t from) {
        const int u = tops.threads[slot / per], i = slot % per;
        if (i == per - 1) {
            if (u < head) add_candidate(tops, key_of(Elem<DT>::widen(x[u]), uint32_t(u)), from);
            if (u < n - tail)
                add_candidate(tops, key_of(Elem<DT>::widen(x[tail + u]), uint32_t(tail + u)), from);
            return;
        }
        const int chunk = u + i * NT;
        if (chunk >= chunks) return;
        const Pack<T, W> one[1] = {load_pack<T, W>(body + int64_t(chunk) * W)};
        add_candidates<DT>(tops, one, (1u << W) - 1, from, [&](int j) { return head + chunk * W + j; });
    };
    select_top(tops, floor, tops.n_threads * per, top, look, emit, found);
}

// ------------------------------------------------------------------ among the beams -----
// Totals as integers of the same order; 0 for those that do not count.
__device__ inline uint64_t ordered64(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
    return x > -__builtin_inf() ? ((b >> 63) ? ~b : b | uint64_t(1) << 63) : 0;
}
__device__ inline float total_value(uint64_t o)
{
    return float(__builtin_bit_cast(double, (o >> 63) ? o & ~(uint64_t(1) << 63) : ~o));
}

// Continuations to be ranked: their totals, and what orders equal ones, the beam and the logit's key.
template <int MOST> struct BeamList {
    uint64_t total[MOST], key[MOST];
    uint8_t beam[MOST];

    __device__ void put(int i, uint64_t t, uint64_t k, int b) { total[i] = t; key[i] = k; beam[i] = uint8_t(b); }
    // how many of the first n come before entry i
    __device__ int rank(int i, int n) const
    {
        const uint64_t t = total[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            if (total[j] > t) ++r;
            else if (total[j] == t)
                r += beam[j] != beam[i] ? beam[j] < beam[i] : key[j] > key[i];
        }
        return r;
    }
};

// One workgroup per request: each beam's log-sum-exp from its parts, then the `top` best of the
// parts' W splits top keys. A bound that at least `top` of them reach comes from the threads' best
// ones; those that reach it are ranked against each other. All of it is latency: the keys are
// loaded first, what fits the registers (kKept to a thread), and meanwhile the sums are joined, the
// parts of several beams side by side. 128 requests of 8 beams, 16 of each: 5 us, of which the way to the
// first loads is a fifth, the sums' logarithms a fifth, bound, list and ranks a fifth each; 2 of 64
// beams in six parts, 64 of each: 68 us, most of it the keys' loads and the totals, taken twice.
constexpr int kChoiceThreads = 256, kKept = 8;
__global__ __launch_bounds__(kChoiceThreads) void k_beam_choice(BeamArgs p)
{
    constexpr int NT = kChoiceThreads, WAVES = NT / 64, SHARE = 64 / WAVES, MOST = 1024;
    // a total is (x - peak) + offset: taken in this order, logits far from 0 cancel first
    __shared__ double offset[BEAM_MAX];                   // score - log of the sum; of a finished beam its score
    __shared__ float peaks[BEAM_MAX];
    __shared__ bool ended[BEAM_MAX];
    __shared__ uint32_t best[NT];
    __shared__ int ranks[NT];
    __shared__ BeamList<MOST> list;
    __shared__ uint64_t kept_total[BEAM_MAX], kept_key[BEAM_MAX];
    __shared__ uint8_t kept_beam[BEAM_MAX];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t request = blockIdx.x, row0 = request * p.W;
    const char *parts = p.parts + row0 * p.splits * p.part_bytes;
    const auto part = [&](int i) { return reinterpret_cast<const RowPart *>(parts + i * p.part_bytes); };
    const int total = p.W * p.splits * p.top;
    // Key i: part i / top's, which are in descending order. Each part starts with another one, or the
    // threads' best ones would be firsts in one thread and lasts in another, and the bound the best of
    // the lasts (with top = 64: 24576 keys of 64 beams took 3.8 ms).
    const auto load_key = [&](int i, int &w) {
        const int at = divide(i, p.by_top), r = i - at * p.top + at - divide(at, p.by_top) * p.top;
        w = divide(at, p.by_splits);
        return reinterpret_cast<const uint64_t *>(part(at) + 1)[r < p.top ? r : r - p.top];
    };
    // lanes to a beam: as many as it has parts, a power of two
    int lanes = 1;
    while (lanes < p.splits && lanes < 64) lanes *= 2;
    const int sub = tid & (lanes - 1), group = tid / lanes;
    // (finished beams have no parts written: what is read of them is not used)
    const auto row_part = [&](int w, int s) { return w < p.W && s < p.splits ? *part(w * p.splits + s) : RowPart{kLowest, 0.0f, 0.0f, 0.0f}; };
    RowPart first = row_part(group, sub);
    double value = group < p.W ? double(p.scores[row0 + group]) : 0.0;
    bool done = group < p.W && p.finished && p.finished[row0 + group];
    uint64_t key[kKept];
    int beam[kKept];
#pragma unroll
    for (int e = 0; e < kKept; ++e) {
        beam[e] = 0;
        key[e] = e * NT + tid < total ? load_key(e * NT + tid, beam[e]) : 0;
    }
    for (int w = group; w < p.W;) {
        float m = kLowest;
        if (!done) {
            m = first.peak;
            for (int s = sub + lanes; s < p.splits; s += lanes) m = __builtin_fmaxf(m, row_part(w, s).peak);
            for (int d = 1; d < lanes; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
            const auto term = [&](const RowPart &q) { return double(q.sum) * double(beam_rescale(q.peak, m)); };
            double sum = term(first);
            for (int s = sub + lanes; s < p.splits; s += lanes) sum += term(row_part(w, s));
            for (int d = 1; d < lanes; d <<= 1) sum += __shfl_xor(sum, d);
            value -= log2(sum) * kNats + (beam_near(m) ? double(m * kLog2e) * kNats - double(m) : 0.0);
        }
        if (sub == 0) { offset[w] = value; peaks[w] = m; ended[w] = done; }
        w += NT / lanes;
        if (w < p.W) {
            first = row_part(w, sub);
            value = double(p.scores[row0 + w]);
            done = p.finished && p.finished[row0 + w];
        }
    }
    if (tid == 0) count = 0;
    __syncthreads();

    // the total of key i, which is beam w's; of a finished beam the first counts alone
    const auto total_of = [&](uint64_t k, int i, int w) -> uint64_t {
        if (ended[w]) return i == w * p.splits * p.top ? ordered64(offset[w]) : 0;
        return k == 0 ? 0 : ordered64((double(key_value(k)) - double(peaks[w])) + offset[w]);
    };
    uint64_t mine = 0, t[kKept];
#pragma unroll
    for (int e = 0; e < kKept; ++e) {
        t[e] = e * NT + tid < total ? total_of(key[e], e * NT + tid, beam[e]) : 0;
        mine = max(mine, t[e]);
    }
    // those that are not kept, kKept loads at a time
    const auto each_further = [&](auto take) __attribute__((always_inline)) {
        for (int i0 = kKept * NT + tid; i0 < total; i0 += kKept * NT) {
            uint64_t k[kKept];
            int w[kKept];
#pragma unroll
            for (int e = 0; e < kKept; ++e) k[e] = load_key(min(i0 + e * NT, total - 1), w[e]);
#pragma unroll
            for (int e = 0; e < kKept; ++e)
                if (i0 + e * NT < total) take(total_of(k[e], i0 + e * NT, w[e]), k[e], w[e]);
        }
    };
    each_further([&](uint64_t t, uint64_t, int) { mine = max(mine, t); });
    best[tid] = uint32_t(mine >> 32);
    __syncthreads();
    // the threads joined to 64; the least of these that fewer than `top` others exceed, by the
    // totals' upper words
    uint32_t k = best[lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) k = max(k, best[w * 64 + lane]);
    int rank = 0;
#pragma unroll
    for (int j = 0; j < SHARE; ++j) rank += uint32_t(__builtin_amdgcn_readlane(k, wave * SHARE + j)) > k;
    ranks[tid] = rank;
    __syncthreads();
    rank = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) rank += ranks[w * 64 + lane];
    uint64_t at = 0;
    for (int r = p.top - 1; at == 0; --r) at = __ballot(rank == r);          // (rank 0 is always there)
    const uint32_t least = __builtin_amdgcn_readlane(k, __builtin_ctzll(at));
    const uint64_t floor = max(uint64_t(least) << 32, uint64_t(1));

    const auto put = [&](uint64_t total, uint64_t key, int w) {
        if (total < floor) return;
        const int to = atomicAdd(&count, 1);
        if (to < MOST) list.put(to, total, key, w);
    };
#pragma unroll
    for (int e = 0; e < kKept; ++e) put(t[e], key[e], beam[e]);
    each_further(put);
    __syncthreads();
    int n = count;
    if (n > MOST) {
        // many equal totals: NT at a time, the list cut to its best whenever it might overflow; from then on
        // only what comes before the last of these is added
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
        bool cut = false;
        const int last = p.top - 1;
        for (int i0 = 0; i0 < total; i0 += NT) {
            if (i0 + tid < total) {
                int w;
                const uint64_t k = load_key(i0 + tid, w), t = total_of(k, i0 + tid, w);
                const bool before = t > kept_total[last] ||
                                    (t == kept_total[last] &&
                                     (w < kept_beam[last] || (w == kept_beam[last] && k > kept_key[last])));
                if (!cut || before) put(t, k, w);
            }
            __syncthreads();
            n = count;
            __syncthreads();                              // all have read it
            if (n <= MOST - NT) continue;
            for (int i = tid; i < n; i += NT) {
                const int r = list.rank(i, n);
                if (r < p.top) { kept_total[r] = list.total[i]; kept_key[r] = list.key[i]; kept_beam[r] = list.beam[i]; }
            }
            __syncthreads();
            if (tid < p.top) list.put(tid, kept_total[tid], kept_key[tid], kept_beam[tid]);
            if (tid == 0) count = p.top;
            n = p.top;
            cut = true;
            __syncthreads();
        }
    }
    if (n > 64) {
        // Ranking takes n^2: the list is cut to what reaches the total of rank `top`, by the upper words. Every
        // wave finds it by halving, the words in its registers (1024 keys of one beam, 64 of them, with the
        // pass: 322 and 41 us).
        uint32_t upper[MOST / 64], least = 0;
#pragma unroll
        for (int e = 0; e < MOST / 64; ++e) upper[e] = e * 64 + lane < n ? uint32_t(list.total[e * 64 + lane] >> 32) : 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t to = least | 1u << bit;
            int reach = 0;
#pragma unroll
            for (int e = 0; e < MOST / 64; ++e) reach += __popcll(__ballot(upper[e] >= to));
            if (reach >= p.top) least = to;
        }
        uint64_t own_total[MOST / NT], own_key[MOST / NT];
        int own_beam[MOST / NT];
#pragma unroll
        for (int e = 0; e < MOST / NT; ++e) {
            const int i = e * NT + tid;
            own_total[e] = i < n ? list.total[i] : 0;
            own_key[e] = i < n ? list.key[i] : 0;
            own_beam[e] = i < n ? list.beam[i] : 0;
        }
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < MOST / NT; ++e)
            if (own_total[e] != 0 && uint32_t(own_total[e] >> 32) >= least)
                list.put(atomicAdd(&count, 1), own_total[e], own_key[e], own_beam[e]);
        __syncthreads();
        n = count;
    }
    const int64_t out = request * p.top;
    const auto write = [&](int r, uint64_t total, uint64_t key, int w) {
        p.out_scores[out + r] = total_value(total);
        p.out_beams[out + r] = w;
        p.out_tokens[out + r] = ended[w] ? p.pad_token : int64_t(key_index(key));
    };
    if (n <= 64) {
        // a lane holds an entry, and each wave compares them with its share of them
        const uint64_t mt = lane < n ? list.total[lane] : 0, mk = lane < n ? list.key[lane] : 0;
        const int mb = lane < n ? list.beam[lane] : 0;
        int r = 0;
        for (int j = wave; j < n; j += WAVES) {
            const uint64_t jt = lane_key(mt, j), jk = lane_key(mk, j);
            const int jb = __builtin_amdgcn_readlane(mb, j);
            r += jt > mt || (jt == mt && (jb < mb || (jb == mb && jk > mk)));
        }
        ranks[tid] = r;
        __syncthreads();
        if (tid < n) {
            r = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) r += ranks[w * 64 + lane];
            if (r < p.top) write(r, mt, mk, mb);
        }
    } else {
        for (int i = tid; i < n; i += NT) {
            const int r = list.rank(i, n);
            if (r < p.top) write(r, list.total[i], list.key[i], list.beam[i]);
        }
    }
    if (tid < p.top && tid >= n) {
        p.out_scores[out + tid] = kNegInf;
        p.out_beams[out + tid] = -1;
        p.out_tokens[out + tid] = -1;
    }
}

// ------------------------------------------------------------------ the states ----------
struct StateArgs {
    const char *src;
    char *dst;
    int64_t src_row, dst_row, src_step1, dst_step1, src_step2, dst_step2, run;
    int columns, blocks;       // chunks of 16 bytes to a row, workgroups to a request
    int chunks, count2;        // chunks to a piece, pieces along the inner dimension
    Divisor by_blocks, by_chunks, by_count2;
};
constexpr int kStates = 32;    // to a launch: the arguments stay below 4 KB
struct ReorderArgs {
    const void *beams;
    int beam_bytes, W, count;
    int first[kStates];        // first workgroup of each state
    StateArgs states[kStates];
};
static_assert(sizeof(ReorderArgs) <= 4096, "kernel arguments");
static_assert(BEAM_MAX <= 64 && kStates <= 64, "a lane for each beam, and for each state");

// A thread takes 16 bytes of the same place of all of a request's rows: it loads what each row is to
// become, then stores it, so that a state may be reordered in place. Rows that stay where they
// are (in place) are left alone. Bound by memory: 256 rows of 4 caches of 8 x 1000 x 128 bf16 in place take
// 232 us (6.2 TB/s of what moves; with stores that stay in the caches 267). Small states by the
// way from the arguments to the indices to the rows (18 of 4 rows, 13 MB: 6.4 us): the state of a
// workgroup is found by all lanes at once, the request's indices are one load, a lane each.
constexpr int kReorderThreads = 256;
template <int MOST>
__global__ __launch_bounds__(kReorderThreads) void k_reorder(ReorderArgs p)
{
    const int group = blockIdx.x, lane = threadIdx.x & 63;
    const int at_state = lane < p.count ? p.first[lane] : 0x7fffffff;
    const int t = __builtin_amdgcn_readfirstlane(__popcll(__ballot(group >= at_state)) - 1);
    const StateArgs &s = p.states[t];
    const int request = divide(group - p.first[t], s.by_blocks);
    const int64_t row0 = int64_t(request) * p.W;
    int from = lane;
    if (lane < p.W) {
        const int64_t b = token_of(p.beams, p.beam_bytes, row0 + lane);
        from = b >= 0 && b < p.W ? int(b) : lane;
    }
    const int column = (group - p.first[t] - request * s.blocks) * kReorderThreads + int(threadIdx.x);
    const int piece = divide(column, s.by_chunks), i = divide(piece, s.by_count2), j = piece - i * s.count2;
    const int64_t at = int64_t(column - piece * s.chunks) * 16;
    const int n = column < s.columns ? int(min(int64_t(16), s.run - at)) : 0;
    const char *src = s.src + row0 * s.src_row + i * s.src_step1 + j * s.src_step2 + at;
    char *dst = s.dst + row0 * s.dst_row + i * s.dst_step1 + j * s.dst_step2 + at;
    const int64_t src_row = s.src_row, dst_row = s.dst_row;
    // the rows that are written
    const uint64_t rows = p.W == 64 ? ~uint64_t(0) : (uint64_t(1) << p.W) - 1;
    const uint64_t moves = rows & (s.src == s.dst ? __ballot(from != lane) : ~uint64_t(0));
    const auto move = [&](auto zero, int off) __attribute__((always_inline)) {
        typedef decltype(zero) T;
        typedef T __attribute__((aligned(1))) anywhere;
        T v[MOST];
        static_for<0, MOST>([&](auto wc) __attribute__((always_inline)) {
            constexpr int w = decltype(wc)::value;
            v[w] = zero;
            if (moves >> w & 1)
                v[w] = *reinterpret_cast<const anywhere *>(src + __builtin_amdgcn_readlane(from, w) * src_row + off);
        });
        static_for<0, MOST>([&](auto wc) __attribute__((always_inline)) {
            constexpr int w = decltype(wc)::value;
            if (moves >> w & 1) __builtin_nontemporal_store(v[w], reinterpret_cast<anywhere *>(dst + w * dst_row + off));
        });
    };
    if (n == 16) move(Bits<16>::type{}, 0);
    else if (n == 8) move(uint64_t(0), 0);
    else
#pragma unroll 1
        for (int k = 0; k < n; ++k) move(uint8_t(0), k);
}

}  // namespace sgemm
