// kernel_beams.hpp -- kernels of beam_search.h: one pass over each beam's row of logits for its
// log-sum-exp and likeliest tokens, the choice among a request's beams, and the reordering of
// states.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "beam_search.h"
#include "kernel_logprobs.hpp"
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
};

// ------------------------------------------------------------------ a beam's row --------
// Running peak m and s = sum 2^((x - m) log2 e). log2 e is taken in two parts: its rounding to FP32
// alone would move log s by up to 1e-7 for flat rows, and which of two beams' tokens comes first hangs
// on such differences. (The sum's other errors are random in sign and average out: 2e-8.)
constexpr float kLog2eLow = 1.925963033500011e-8f;
struct BeamStats {
    float m = kLowest, s = 0.0f;

    __device__ static float power(float t)             // e^t, t <= 0
    {
        return __builtin_amdgcn_exp2f(__builtin_fmaf(t, kLog2e, t * kLog2eLow));
    }
    __device__ void raise(float to)
    {
        const float next = __builtin_fmaxf(m, to);
        s *= power(__builtin_fmaxf(m - next, -1000.0f));
        m = next;
    }
    // x with m already raised to it
    __device__ void add(float x) { s += power(x - m); }
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
// tid + NT, ... of 16 bytes, up to one of the tail.
template <int DT, int NT, int U, bool STREAM>
__global__ __launch_bounds__(NT) void k_beam_pass(BeamArgs p)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
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
    // the best group: its value in key order, and its first element
    uint32_t best = 0;
    int best_at = tid < head ? tid : tid < chunks ? head + tid * W : tail + tid;
    const bool empty = best_at >= n;
    auto note = [&](float peak, int at) __attribute__((always_inline)) {
        const uint32_t o = ordered(peak);
        best_at = o > best ? at : best_at;
        best = max(best, o);
    };
    float edge[2] = {0.0f, 0.0f};                         // the thread's head and tail elements
    auto take1 = [&](int at, float &v) __attribute__((always_inline)) {
        v = Elem<DT>::widen(x[at]);
        note(v, at);
        st.raise(v);
        st.add(v);
    };
    auto load = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            b[u] = load_chunk_of<STREAM, T, W>(body + int64_t(min(c + u * NT, chunks - 1)) * W);
    };
    auto widen = [&](float (&v)[W], int u, int c) __attribute__((always_inline)) {
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
        float v[U][W], peak = kNegInf;
        load(c);
#pragma unroll
        for (int u = 0; u < U; ++u) peak = __builtin_fmaxf(peak, widen(v[u], u, c));
        st.raise(peak);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j) st.add(v[u][j]);
    }
    if (c < chunks) {                                     // fewer than U are left
        load(c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u * NT >= chunks) break;
            float v[W];
            st.raise(widen(v, u, c));
#pragma unroll
            for (int j = 0; j < W; ++j) st.add(v[j]);
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
    if (chunks <= U * NT) {                               // b holds all of this thread's chunks
        static_assert(U * W <= 32, "a bit for each element");
        if (mine >= floor) {
            const int mine_n = tid < chunks ? (chunks - tid + NT - 1) / NT * W : 0;
            add_candidates<DT>(tops, b, mine_n == 32 ? 0xffffffffu : (1u << mine_n) - 1, floor,
                               [&](int i) { return head + (tid + i / W * NT) * W + i % W; });
            if (tid < head) add_candidate(tops, key_of(edge[0], uint32_t(tid)), floor);
            if (tid < n - tail) add_candidate(tops, key_of(edge[1], uint32_t(tail + tid)), floor);
        }
        __syncthreads();
        const int found = tops.n_cand;
        if (found <= kCandidates) {
            rank_top(tops, found, top, emit);
            return;
        }
        __syncthreads();                                  // all have read it
        if (tid == 0) tops.n_cand = 0;
    }
    if (mine >= floor) tops.threads[atomicAdd(&tops.n_threads, 1)] = tid;
    __syncthreads();
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
    select_top(tops, floor, tops.n_threads * per, top, look, emit);
}

// ------------------------------------------------------------------ among the beams -----
// A continuation: its total, as an integer of the same order (0: it does not count), and what
// orders equal totals, the beam and the logit's key.
struct BeamChoice {
    uint64_t total, key;
    uint32_t beam;
};
__device__ inline uint64_t ordered64(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
    return x > -__builtin_inf() ? ((b >> 63) ? ~b : b | uint64_t(1) << 63) : 0;
}
__device__ inline float total_value(uint64_t o)
{
    return float(__builtin_bit_cast(double, (o >> 63) ? o & ~(uint64_t(1) << 63) : ~o));
}
__device__ inline bool before(const BeamChoice &a, const BeamChoice &b)
{
    if (a.total != b.total) return a.total > b.total;
    return a.beam != b.beam ? a.beam < b.beam : a.key > b.key;
}

// One workgroup per request: each beam's log-sum-exp from its parts, then the `top` best of the
// parts' W splits top keys. A bound that at least `top` of them reach comes from the threads' best
// ones; those that reach it are ranked against each other.
constexpr int kChoiceThreads = 256;
__global__ __launch_bounds__(kChoiceThreads) void k_beam_choice(BeamArgs p)
{
    constexpr int NT = kChoiceThreads, MOST = 1024;
    // a total is (x - peak) + offset: taken in this order, logits far from 0 cancel first
    __shared__ double offset[BEAM_MAX];                   // score - log sum; of a finished beam its score
    __shared__ float peak[BEAM_MAX];
    __shared__ bool ended[BEAM_MAX];
    __shared__ uint64_t best[NT], bound;
    __shared__ BeamChoice list[MOST], kept[64];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t request = blockIdx.x, row0 = request * p.W;
    const char *parts = p.parts + row0 * p.splits * p.part_bytes;
    const auto part = [&](int i) { return reinterpret_cast<const RowPart *>(parts + i * p.part_bytes); };
    for (int w = wave; w < p.W; w += NT / 64) {
        const bool done = p.finished && p.finished[row0 + w];
        double value = double(p.scores[row0 + w]);
        float m = kLowest;
        if (!done) {
            for (int s = lane; s < p.splits; s += 64) m = __builtin_fmaxf(m, part(w * p.splits + s)->peak);
            m = wave_reduce(m, [](float a, float b) { return __builtin_fmaxf(a, b); });
            double sum = 0.0;
            for (int s = lane; s < p.splits; s += 64) {
                const RowPart *q = part(w * p.splits + s);
                sum += double(q->sum) * exp(double(q->peak) - double(m));
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
            value -= log(sum);
        }
        if (lane == 0) { offset[w] = value; peak[w] = m; ended[w] = done; }
    }
    if (tid == 0) { count = 0; bound = 0; }
    __syncthreads();

    const int total = p.W * p.splits * p.top;
    const auto choice = [&](int i) {
        const int at = i / p.top, w = at / p.splits;
        BeamChoice c{0, 0, uint32_t(w)};
        if (ended[w]) {
            if (i == w * p.splits * p.top) c.total = ordered64(offset[w]);
        } else {
            c.key = reinterpret_cast<const uint64_t *>(part(at) + 1)[i - at * p.top];
            if (c.key != 0) c.total = ordered64((double(key_value(c.key)) - double(peak[w])) + offset[w]);
        }
        return c;
    };
    uint64_t mine = 0;
#pragma unroll 4
    for (int i = tid; i < total; i += NT) mine = max(mine, choice(i).total);
    best[tid] = mine;
    __syncthreads();
    if (tid < 64) {
        // the least of the joined lanes' bests that fewer than `top` others exceed
        uint64_t k = best[tid];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) k = max(k, best[w * 64 + tid]);
        int rank = 0;
        for (int j = 0; j < 64; ++j) rank += lane_key(k, j) > k;
        uint64_t t = rank < p.top ? k : ~uint64_t(0);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) t = min(t, uint64_t(__shfl_xor(static_cast<unsigned long long>(t), d)));
        if (tid == 0) bound = max(t, uint64_t(1));
    }
    __syncthreads();
    const uint64_t floor = bound;
    for (int i = tid; i < total; i += NT) {
        const BeamChoice c = choice(i);
        if (c.total < floor) continue;
        const int to = atomicAdd(&count, 1);
        if (to < MOST) list[to] = c;
    }
    __syncthreads();
    int n = count;
    const auto ranked = [&](int have, auto fn) {
        for (int i = tid; i < have; i += NT) {
            const BeamChoice c = list[i];
            int r = 0;
            for (int j = 0; j < have; ++j) r += before(list[j], c);
            if (r < p.top) fn(r, c);
        }
    };
    if (n > MOST) {
        // many equal totals: NT at a time, the list cut to its best whenever it might overflow
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
        for (int i0 = 0; i0 < total; i0 += NT) {
            if (i0 + tid < total) {
                const BeamChoice c = choice(i0 + tid);
                if (c.total >= floor) list[atomicAdd(&count, 1)] = c;
            }
            __syncthreads();
            n = count;
            __syncthreads();                              // all have read it
            if (n <= MOST - NT) continue;
            ranked(n, [&](int r, const BeamChoice &c) { kept[r] = c; });
            __syncthreads();
            if (tid < p.top) list[tid] = kept[tid];
            if (tid == 0) count = p.top;
            n = p.top;
            __syncthreads();
        }
    }
    const int64_t out = request * p.top;
    ranked(n, [&](int r, const BeamChoice &c) {
        p.out_scores[out + r] = total_value(c.total);
        p.out_beams[out + r] = int64_t(c.beam);
        p.out_tokens[out + r] = ended[c.beam] ? p.pad_token : int64_t(key_index(c.key));
    });
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
    int count2, chunks;        // pieces along the inner dimension, chunks of 16 bytes to a piece
    int columns, blocks;       // chunks to a row, workgroups to a request
};
constexpr int kStates = 40;    // to a launch: the arguments stay below 4 KB
struct ReorderArgs {
    const void *beams;
    int beam_bytes, W, count;
    int first[kStates];        // first workgroup of each state
    StateArgs states[kStates];
};
static_assert(sizeof(ReorderArgs) <= 4096, "kernel arguments");

// A thread takes 16 bytes of the same place of all of a request's rows: it loads what each row is to
// become, then stores it, so that a state may be reordered in place. Rows that stay where they
// are (in place) are left alone.
constexpr int kReorderThreads = 256;
template <int MOST>
__global__ __launch_bounds__(kReorderThreads) void k_reorder(ReorderArgs p)
{
    const int group = blockIdx.x;
    int t = 0;
    while (t + 1 < p.count && group >= p.first[t + 1]) ++t;
    const StateArgs &s = p.states[t];
    const int request = (group - p.first[t]) / s.blocks;
    const int column = (group - p.first[t] - request * s.blocks) * kReorderThreads + int(threadIdx.x);
    if (column >= s.columns) return;
    const int piece = column / s.chunks, i = piece / s.count2, j = piece - i * s.count2;
    const int64_t at = int64_t(column - piece * s.chunks) * 16;
    const int n = int(min(int64_t(16), s.run - at));
    const int64_t row0 = int64_t(request) * p.W;
    const char *src = s.src + row0 * s.src_row + i * s.src_step1 + j * s.src_step2 + at;
    char *dst = s.dst + row0 * s.dst_row + i * s.dst_step1 + j * s.dst_step2 + at;
    const bool in_place = s.src == s.dst;
    int from[MOST];
#pragma unroll
    for (int w = 0; w < MOST; ++w) {
        from[w] = w;
        if (w < p.W) {
            const int64_t b = token_of(p.beams, p.beam_bytes, row0 + w);
            if (b >= 0 && b < p.W) from[w] = __builtin_amdgcn_readfirstlane(int(b));
        }
    }
    const auto move = [&](auto zero, int off) __attribute__((always_inline)) {
        typedef Pack<decltype(zero), 1> P;
        P v[MOST];
#pragma unroll
        for (int w = 0; w < MOST; ++w)
            if (w < p.W && !(in_place && from[w] == w))
                v[w] = *reinterpret_cast<const P *>(src + from[w] * s.src_row + off);
#pragma unroll
        for (int w = 0; w < MOST; ++w)
            if (w < p.W && !(in_place && from[w] == w))
                *reinterpret_cast<P *>(dst + w * s.dst_row + off) = v[w];
    };
    if (n == 16) { move(Bits<16>::type{}, 0); return; }
    if (n & 8) move(uint64_t(0), 0);
    if (n & 4) move(uint32_t(0), n & 8);
    if (n & 2) move(uint16_t(0), n & 12);
    if (n & 1) move(uint8_t(0), n & 14);
}

}  // namespace sgemm
