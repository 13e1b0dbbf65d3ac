// kernel_logprobs.hpp -- kernels of token_logprobs.h: one pass over each row of logits for
// its log-sum-exp, entropy and top alternatives, the join of rows that were split, and the
// gradient.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ops_common.hpp"

namespace sgemm {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e38f;

// A row part's result in the workspace: `top` keys follow, in descending order.
struct RowPart {
    float peak;      // the largest logit (as kept by RowStats)
    float sum;       // sum of 2^((x - peak) log2 e)
    float dot;       // sum of (x - peak) log2 e times the same
    float pad;
};

struct RowArgs {
    const void *logits;
    int64_t ld;
    const void *tokens;
    float *logprobs, *entropy, *lse, *lse_low, *top_logprobs;
    int64_t *top_tokens;
    char *parts;          // splits > 1: part s of row i at (i * splits + s) * part_bytes
    int64_t part_bytes;
    int M, V, top, splits, part_len, token_bytes;
};

__device__ inline int64_t token_of(const void *tokens, int bytes, int64_t row)
{
    return bytes == 8 ? static_cast<const int64_t *>(tokens)[row]
                      : int64_t(static_cast<const int32_t *>(tokens)[row]);
}

// ------------------------------------------------------------------ a row's sums --------
// Running peak m, s = sum e and d = sum y e with y = (x - m) log2 e and e = 2^y, in base 2
// so that e is one hardware instruction. When m grows by g (in base-2 units, g >= 0) every
// y falls by g: s' = s 2^-g, d' = (d - g s) 2^-g. The entropy in nats is then
// log s - ln2 d / s, a sum of two terms of one sign: nothing cancels. m is kept finite from
// below (kLowest), so a row of -infinity has y = -infinity and s = 0, and y e is taken with
// y at least -1000, where e is 0 already.
struct RowStats {
    float m = kLowest, s = 0.0f, d = 0.0f;

    __device__ void raise(float to)
    {
        const float next = __builtin_fmaxf(m, to);
        const float g = __builtin_fmaxf((m - next) * kLog2e, -1000.0f);
        const float f = __builtin_amdgcn_exp2f(g);
        d = (d + g * s) * f;
        s = s * f;
        m = next;
    }
    // x with m already raised to it
    __device__ void add(float x)
    {
        const float y = (x - m) * kLog2e;
        const float e = __builtin_amdgcn_exp2f(y);
        s += e;
        d = __builtin_fmaf(__builtin_fmaxf(y, -1000.0f), e, d);
    }
    __device__ void join(float m2, float s2, float d2)
    {
        const float next = __builtin_fmaxf(m, m2);
        const float g = __builtin_fmaxf((m2 - next) * kLog2e, -1000.0f);
        raise(next);
        const float f = __builtin_amdgcn_exp2f(g);
        d += (d2 + g * s2) * f;
        s += s2 * f;
    }
};

// ------------------------------------------------------------------ the alternatives ----
// Elements in a total order as 64-bit keys: the value's bits mapped to unsigned integers of
// the same order (NaN lowest, -0 as +0), then the index, lower ones first. Keys are
// distinct and never 0.
__device__ inline uint32_t ordered(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ inline uint64_t key_of(float x, uint32_t index)
{
    return uint64_t(ordered(x)) << 32 | (0xffffffffu - index);
}
__device__ inline float key_value(uint64_t key)
{
    const uint32_t o = uint32_t(key >> 32);
    const uint32_t b = (o & 0x80000000u) ? o & 0x7fffffffu : ~o;
    return o == 0 ? __builtin_nanf("") : __builtin_bit_cast(float, b);
}
__device__ inline uint32_t key_index(uint64_t key) { return 0xffffffffu - uint32_t(key); }

__device__ inline uint64_t lane_key(uint64_t key, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(key), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(key >> 32), lane);
    return uint64_t(hi) << 32 | lo;
}

// The `top` largest of many keys, by a bound and a short list of candidates.
//  * The elements lie in groups of neighbours (a chunk of one load); each thread knows the
//    best key of its groups, key_of(largest value, first index of the first group that holds
//    it). Of two groups' keys the larger belongs to the group whose best element is larger.
//  * top_bound(): the threads' bests are joined to 64, and T is the top-th largest of those:
//    exact for top = 1, about 24 elements reach it for top = 20. At least `top` threads hold a
//    group whose key is T or more, so elements of a group below T, and elements below T's value
//    or equal to it behind its group, are not among the top ones.
//  * The elements of the threads whose best reaches T become candidates where they reach it
//    themselves: from registers where the row fits them, else looked at again, by all threads
//    in turn. With the keys in no order there are little more than `top`; each is ranked
//    against all. Rows made to defeat the bound bring more: the list is cut to the `top` best
//    whenever it could overflow, and T rises to the last of them.
// All of this runs once a row, behind the pass, so latency is what counts: 1 x 131072 f32 with 20
// alternatives takes 9.4 us in both kernels (9.0 with the selections left out), 600 x 50001 bf16
// with 5 takes 21.0 (15.6 without). Candidates kept on the way, above a T of the row's first
// elements, save the second look, but the wait for that T costs more wherever rows share a
// compute unit (1200 x 32000 bf16, 20: 38 us instead of 23.6). Ranking 64 keys in one wave costs
// 1.7 us a row, shared among the waves 0.7.
constexpr int kCandidates = 1024, kNarrow = 64;
template <int NT> struct TopShared {
    uint64_t best[NT], joined[NT];
    uint64_t cand[kCandidates], kept[64];
    int ranks[NT], threads[NT];
    int n_threads, n_cand;
};

// T, 0 where fewer than `top` of the 64 joined threads have elements. best is 0 for a thread
// without. Every wave joins all of them and compares them with its share of them.
template <int NT>
__device__ inline uint64_t top_bound(TopShared<NT> &sh, uint64_t best, int top)
{
    constexpr int WAVES = NT / 64, SHARE = 64 / WAVES;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    sh.best[tid] = best;
    __syncthreads();
    uint64_t k = sh.best[lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) k = max(k, sh.best[w * 64 + lane]);
    sh.joined[tid] = k;
    __builtin_amdgcn_wave_barrier();
    const uint64_t *others = sh.joined + wave * 64 + wave * SHARE;
    int rank = 0;
#pragma unroll
    for (int j = 0; j < SHARE; ++j) rank += others[j] > k;
    sh.ranks[tid] = rank;
    __syncthreads();
    rank = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) rank += sh.ranks[w * 64 + lane];
    // keys but 0 are distinct; with fewer than `top` of them none has this rank, or a 0 has
    const uint64_t at = __ballot(rank == top - 1);
    return at == 0 ? 0 : lane_key(k, __builtin_ctzll(at));
}

// Ranks the candidates; fn(rank, key) for those among the top.
template <int NT, typename Fn>
__device__ inline void rank_candidates(const TopShared<NT> &sh, int n, int top, Fn fn)
{
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t k = sh.cand[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > k;
        if (rank < top) fn(rank, k);
    }
}

template <int NT> __device__ inline void add_candidate(TopShared<NT> &sh, uint64_t key, uint64_t floor)
{
    if (key < floor) return;
    const int to = atomicAdd(&sh.n_cand, 1);
    if (to < kCandidates) sh.cand[to] = key;
}

// The elements of chunks b[u], u < U, that reach floor join the candidates; at(i) is the index of
// element i of them, `there` has a bit for each that exists. The few that do are taken one
// after another, picked from the registers: code that runs once a row is short, for its
// instructions come from memory.
template <int DT, int NT, int U, int W, typename At>
__device__ inline void add_candidates(TopShared<NT> &sh, const Pack<typename Elem<DT>::type, W> (&b)[U],
                                      uint32_t there, uint64_t floor, At at)
{
    typedef typename Elem<DT>::type T;
    const float least = key_value(floor);          // not a number where NaNs reach it
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < U * W; ++i)
        hits |= Elem<DT>::widen(b[i / W].v[i % W]) < least ? 0u : 1u << i;
    hits &= there;
    while (hits != 0) {
        const int i = __builtin_ctz(hits);
        hits &= hits - 1;
        T x = b[0].v[0];
#pragma unroll
        for (int k = 1; k < U * W; ++k) x = i == k ? b[k / W].v[k % W] : x;
        add_candidate(sh, key_of(Elem<DT>::widen(x), uint32_t(at(i))), floor);
    }
}

// The top of the n <= kCandidates candidates, all of them in the list behind a barrier.
template <int NT, typename Emit>
__device__ inline void rank_top(TopShared<NT> &sh, int n, int top, Emit emit)
{
    if (n > 96) {                              // cut the list first: ranking takes n^2
        constexpr int EACH = (kCandidates + NT - 1) / NT;
        uint64_t mine[EACH], best = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = i * NT + int(threadIdx.x);
            mine[i] = at < n ? sh.cand[at] : 0;
            best = max(best, mine[i]);
        }
        const uint64_t t = top_bound(sh, best, top);
        if (threadIdx.x == 0) sh.n_cand = 0;
        __syncthreads();
        int more = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) more += mine[i] != 0 && mine[i] >= t;
        if (more != 0) {
            int to = atomicAdd(&sh.n_cand, more);
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (mine[i] != 0 && mine[i] >= t) sh.cand[to++] = mine[i];
        }
        __syncthreads();
        n = sh.n_cand;
    }
    rank_candidates(sh, n, top, emit);
}

// look(slot, floor) adds what reaches floor among the at most 8 elements of a slot to the
// candidates. All slots, NT at a time; where that brings more than the list holds, again
// kNarrow at a time from a list cut to the top. Then emit(rank, key) for the top.
template <int NT, typename Look, typename Emit>
__device__ inline void select_top(TopShared<NT> &sh, uint64_t floor, int slots, int top, Look look,
                                  Emit emit)
{
    static_assert(kCandidates >= 2 * kNarrow * 8, "the list holds a narrow step");
    int width = NT, have = 0;
    for (int at = 0; at < slots;) {
        const int slot = at + int(threadIdx.x);
        if (int(threadIdx.x) < width && slot < slots) look(slot, floor);
        __syncthreads();
        const int n = sh.n_cand;
        const bool fits = n <= kCandidates;
        if (fits) { at += width; have = n; }
        else width = kNarrow;                  // and this step again
        if (at >= slots) break;
        __syncthreads();                       // all have read n before it changes
        if (!fits || n > kCandidates - kNarrow * 8) {
            if (have > top) {
                rank_candidates(sh, have, top, [&](int r, uint64_t k) { sh.kept[r] = k; });
                __syncthreads();
                if (int(threadIdx.x) < top) sh.cand[threadIdx.x] = sh.kept[threadIdx.x];
                floor = max(floor, sh.kept[top - 1]);
                have = top;
            }
            if (threadIdx.x == 0) sh.n_cand = have;
            __syncthreads();
        }
    }
    rank_top(sh, have, top, emit);
}

// ------------------------------------------------------------------ joining lanes -------
template <int NT> struct StatsShared {
    float m[NT / 64], s[NT / 64], d[NT / 64];
};

// A reduction over the wave's lanes in a fixed order: cross-lane moves inside rows of 16, then
// the four rows. Every lane gets the result.
template <int CTRL> __device__ inline float lane_moved(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                                 0xf, 0xf, true));
}
template <typename Op> __device__ inline float wave_reduce(float x, Op op)
{
    x = op(x, lane_moved<0xb1>(x));          // lane ^ 1
    x = op(x, lane_moved<0x4e>(x));          // lane ^ 2
    x = op(x, lane_moved<0x141>(x));         // the other four of eight
    x = op(x, lane_moved<0x140>(x));         // the other eight of 16
    auto row = [&](int r) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * r));
    };
    return op(op(row(0), row(1)), op(row(2), row(3)));
}

// Every thread gets the workgroup's joined sums (in the same order each time): the lanes are
// brought to their largest peak first, then summed.
template <int NT> __device__ inline RowStats join_stats(StatsShared<NT> &sh, RowStats st)
{
    const auto larger = [](float a, float b) { return __builtin_fmaxf(a, b); };
    const auto plus = [](float a, float b) { return a + b; };
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    st.raise(wave_reduce(st.m, larger));
    st.s = wave_reduce(st.s, plus);
    st.d = wave_reduce(st.d, plus);
    if (lane == 0) { sh.m[wave] = st.m; sh.s[wave] = st.s; sh.d[wave] = st.d; }
    __syncthreads();
    RowStats all;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) all.m = __builtin_fmaxf(all.m, sh.m[w]);
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        RowStats one;
        one.m = sh.m[w]; one.s = sh.s[w]; one.d = sh.d[w];
        one.raise(all.m);
        all.s += one.s;
        all.d += one.d;
    }
    return all;
}

// The row's token and its logit, loaded ahead of the sums.
struct RowToken {
    int64_t t;
    float x;
};
template <int DT> __device__ inline RowToken load_token(const RowArgs &p, int64_t row)
{
    typedef typename Elem<DT>::type T;
    const int64_t t = token_of(p.tokens, p.token_bytes, row);
    return {t, t >= 0 && t < p.V
                   ? Elem<DT>::widen(static_cast<const T *>(p.logits)[row * p.ld + t]) : 0.0f};
}

__device__ inline void write_row(const RowArgs &p, int64_t row, const RowStats &st, RowToken token)
{
    const bool none = st.s == 0.0f;                       // nothing but -infinity
    const float logs = __builtin_logf(st.s);
    // x - m is small where x is likely, so it is taken before log s is
    float lp = none ? kNegInf : (token.x - st.m) - logs;
    if (token.t >= p.V) lp = __builtin_nanf("");
    p.logprobs[row] = token.t < 0 ? 0.0f : lp;
    if (p.entropy) p.entropy[row] = none ? 0.0f : logs - kLn2 * (st.d / st.s);
    const float lse = none ? kNegInf : st.m + logs;
    if (p.lse) p.lse[row] = lse;
    if (p.lse_low) {
        // m + log s - lse without rounding (the terms of a sum's error, for either order of size)
        const float part = lse - st.m;
        const float low = (st.m - (lse - part)) + (logs - part);
        p.lse_low[row] = none || __builtin_fabsf(lse) < 64.0f ? 0.0f : low;
    }
}
__device__ inline void write_top(const RowArgs &p, int64_t row, const RowStats &st, int r,
                                 uint64_t key)
{
    const float x = key_value(key);
    p.top_logprobs[row * p.top + r] =
        st.s == 0.0f ? (x == x ? kNegInf : x) : (x - st.m) - __builtin_logf(st.s);
    p.top_tokens[row * p.top + r] = key_index(key);
}

template <bool STREAM, typename T, int W> __device__ inline Pack<T, W> load_chunk_of(const T *p)
{
    if constexpr (STREAM) return load_pack_stream<T, W>(p);
    else return load_pack<T, W>(p);
}

// ------------------------------------------------------------------ the pass ------------
// One workgroup per (row, part). A thread's elements: up to one of the head before the
// first 16-byte boundary, then the chunks tid, tid + NT, ... of 16 bytes, then up to one
// of the tail. U chunks are in flight, and the peak is raised once for them. HBM-bound where
// rows fill the card: 4096 x 131072 bf16 takes 165 us (6.5 TB/s) with STREAM, loads that do not
// stay in the caches, and 188 without; where the logits fit the caches, STREAM costs (511 x 32001
// f32 12.4 to 12.8 us).
template <int DT, bool TOP, int NT, int U, bool STREAM>
__global__ __launch_bounds__(NT) void k_row_pass(RowArgs p)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    __shared__ StatsShared<NT> stats;
    __shared__ TopShared<TOP ? NT : 64> tops;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / p.splits;
    const int part = blockIdx.x % p.splits;
    const int first = part * p.part_len;                  // this part's elements of the row
    const int n = min(p.part_len, p.V - first);
    const T *x = static_cast<const T *>(p.logits) + row * p.ld + first;
    const int head = min(n, int((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
    const int chunks = (n - head) / W;
    const int tail = head + chunks * W;                   // first element of the tail
    const T *body = x + head;
    RowToken token{};
    // the row's results are the last wave's to write, while the others go on to the alternatives
    if (p.splits == 1 && tid == NT - 1) token = load_token<DT>(p, row);
    if (TOP && tid == 0) { tops.n_cand = 0; tops.n_threads = 0; }

    RowStats st;
    Pack<T, W> b[U];
    // the best group: its value in key order, and its first element
    uint32_t best = 0;
    int best_at = tid < head ? tid : tid < chunks ? head + tid * W : tail + tid;
    const bool empty = best_at >= n;
    auto note = [&](float peak, int at) __attribute__((always_inline)) {
        if constexpr (TOP) {
            const uint32_t o = ordered(peak);
            best_at = o > best ? at : best_at;
            best = max(best, o);
        }
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

    const RowStats all = join_stats(stats, st);           // a barrier: the candidates are there
    RowPart *out = reinterpret_cast<RowPart *>(p.parts + int64_t(blockIdx.x) * p.part_bytes);
    if (tid == NT - 1) {
        if (p.splits == 1) write_row(p, row, all, token);
        else *out = RowPart{all.m, all.s, all.d, 0.0f};
    }
    if constexpr (TOP) {
        uint64_t *keys = reinterpret_cast<uint64_t *>(out + 1);
        auto emit = [&](int r, uint64_t k) {
            if (p.splits > 1) keys[r] = k - uint32_t(first);     // indices in the row
            else write_top(p, row, all, r, k);
        };
        // a part shorter than `top` leaves its last keys empty
        if (p.splits > 1 && tid < p.top && tid >= n) keys[tid] = 0;
        const uint64_t mine = empty ? 0 : uint64_t(best) << 32 | (0xffffffffu - uint32_t(best_at));
        uint64_t floor = top_bound(tops, mine, p.top);
        // T's group reaches W - 1 elements behind its first
        floor = max(floor - min(uint32_t(floor), uint32_t(W - 1)), uint64_t(1));
        if (chunks <= U * NT) {                           // b holds all of this thread's chunks
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
                rank_top(tops, found, p.top, emit);
                return;
            }
            __syncthreads();                              // all have read it
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
            const Pack<T, W> c[1] = {load_pack<T, W>(body + int64_t(chunk) * W)};
            add_candidates<DT>(tops, c, (1u << W) - 1, from, [&](int j) { return head + chunk * W + j; });
        };
        select_top(tops, floor, tops.n_threads * per, p.top, look, emit);
    }
}

// Joins a row's parts: the sums in one order of the parts, the alternatives from the parts'
// lists (every key is a group of its own).
template <int DT, bool TOP>
__global__ __launch_bounds__(256) void k_row_join(RowArgs p)
{
    constexpr int NT = 256, EACH = 4;
    static_assert(EACH * NT <= kCandidates, "the list holds every key");
    __shared__ StatsShared<NT> stats;
    __shared__ TopShared<TOP ? NT : 64> tops;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const char *parts = p.parts + row * p.splits * p.part_bytes;
    RowToken token{};
    if (tid == NT - 1) token = load_token<DT>(p, row);
    if (TOP && tid == 0) tops.n_cand = 0;
    const int n = TOP ? p.splits * p.top : 0;
    auto key_at = [&](int i) {
        const int s = i / p.top;
        return reinterpret_cast<const uint64_t *>(parts + s * p.part_bytes +
                                                  sizeof(RowPart))[i - s * p.top];
    };
    uint64_t mine[EACH], best = 0;                        // the first keys; often they are all
    if constexpr (TOP) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            mine[i] = tid + i * NT < n ? key_at(tid + i * NT) : 0;
            best = max(best, mine[i]);
        }
        for (int i = tid + EACH * NT; i < n; i += NT) best = max(best, key_at(i));
    }
    RowStats st;
    for (int s = tid; s < p.splits; s += NT) {
        const RowPart *q = reinterpret_cast<const RowPart *>(parts + s * p.part_bytes);
        st.join(q->peak, q->sum, q->dot);
    }
    const RowStats all = join_stats(stats, st);
    if (tid == NT - 1) write_row(p, row, all, token);
    if constexpr (TOP) {
        const uint64_t floor = max(top_bound(tops, best, p.top), uint64_t(1));
        auto emit = [&](int r, uint64_t k) { write_top(p, row, all, r, k); };
        if (n <= EACH * NT) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                add_candidate(tops, mine[i], floor);
            __syncthreads();
            rank_top(tops, tops.n_cand, p.top, emit);
        } else {
            select_top(tops, floor, n, p.top,
                       [&](int slot, uint64_t least) { add_candidate(tops, key_at(slot), least); },
                       emit);
        }
    }
}

// ------------------------------------------------------------------ the gradient --------
struct GradArgs {
    const void *logits;
    void *grad;
    const void *tokens;
    const float *lse, *lse_low, *entropy, *g_logprob, *g_entropy, *g_lse;
    int64_t ld, ldg;
    int M, V, token_bytes, parts, part_len;
};

// One workgroup per (row, part): dx = -p (a + h (logp + H)), plus g at the token, with
// a = g - g_lse and h = g_entropy. HBM-bound: 4096 x 131072 bf16 with the entropy's term takes 362 us
// (5.9 TB/s, reading and writing; a large copy reaches 4.8), 511 x 32001 f32 22.3.
constexpr int kGradThreads = 256;
template <int DT, bool STREAM>
__global__ __launch_bounds__(kGradThreads) void k_row_gradient(GradArgs p)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / p.parts;
    const int first = int(blockIdx.x % p.parts) * p.part_len;
    const int n = min(p.part_len, p.V - first);
    const T *x = static_cast<const T *>(p.logits) + row * p.ld + first;
    T *out = static_cast<T *>(p.grad) + row * p.ldg + first;

    const int64_t t = token_of(p.tokens, p.token_bytes, row);
    float lse = p.lse[row];
    const float low = p.lse_low ? p.lse_low[row] : 0.0f;
    float g = p.g_logprob && t >= 0 ? p.g_logprob[row] : 0.0f;
    float h = p.g_entropy ? p.g_entropy[row] : 0.0f;
    const float entropy = p.g_entropy ? p.entropy[row] : 0.0f;
    float a = g - (p.g_lse ? p.g_lse[row] : 0.0f);
    if (t >= p.V && p.g_logprob) a = __builtin_nanf("");
    if (lse == kNegInf) { lse = 0.0f; g = 0.0f; a = 0.0f; h = 0.0f; }   // p = 0 throughout
    const int64_t at = t - first;                         // the token's element of the part
    auto value = [&](float v, bool is_token) __attribute__((always_inline)) {
        const float logp = (v - lse) - low;
        const float pr = __builtin_amdgcn_exp2f(logp * kLog2e);
        const float w = __builtin_fmaf(h, __builtin_fmaxf(logp, -1000.0f) + entropy, a);
        const float dx = -pr * w;
        return is_token ? dx + g : dx;
    };
    const int head = min(n, int((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
    const int chunks = (n - head) / W;
    const int tail = head + chunks * W;
    if (tid < head) out[tid] = Elem<DT>::narrow(value(Elem<DT>::widen(x[tid]), tid == at));
    if (tid < n - tail)
        out[tail + tid] = Elem<DT>::narrow(value(Elem<DT>::widen(x[tail + tid]), tail + tid == at));
    // the token's chunk and its place there, -1 if it is none of this part's
    const int body = int(at < head || at >= tail ? -W : at - head);
    const int token_chunk = body < 0 ? -1 : body / W, place = body % W;
    for (int c = tid; c < chunks; c += kGradThreads) {
        const int64_t e = head + int64_t(c) * W;
        const Pack<T, W> in = load_chunk_of<STREAM, T, W>(x + e);
        float v[W];
        Pack<T, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = value(Elem<DT>::widen(in.v[j]), false);
        if (c == token_chunk) {
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] += j == place ? g : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) o.v[j] = Elem<DT>::narrow(v[j]);
        store_pack_stream(out + e, o);
    }
}

}  // namespace sgemm
