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
    float *logprobs, *entropy, *lse, *top_logprobs;
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

// The `top` largest of many keys, by a bound and a short list of candidates.
//  * The elements lie in groups of neighbours (a chunk of one load); each thread knows the
//    best key of its groups, key_of(largest value, first index of the first group that holds
//    it). Of two groups' keys the larger belongs to the group whose best element is larger.
//  * bound(): a wave takes the n-th largest of its threads' bests, n = ceil(top / waves); the
//    smallest of those is T. At least `top` threads hold a group whose key is T or more, so
//    elements of a group below T, and elements below T's value or equal to it behind its
//    group, are not among the top ones.
//  * The threads whose best reaches T (about `top` of them) have their elements looked at
//    again, by all threads in turn, and the elements that reach T become candidates. With
//    the keys in no order there are little more than `top`; each is ranked against all.
//    Rows made to defeat the bound bring more: the list is cut to the `top` best whenever it
//    could overflow, and T rises to the last of them.
constexpr int kCandidates = 1024, kNarrow = 64;
template <int NT> struct TopShared {
    uint64_t best[NT];
    uint64_t cand[kCandidates], kept[64];
    uint64_t least[NT / 64];
    int threads[NT];
    int n_threads, n_cand;
};

// T, and the threads that reach it in sh.threads. best is 0 for a thread without elements.
template <int NT>
__device__ inline uint64_t top_bound(TopShared<NT> &sh, uint64_t best, int top)
{
    constexpr int WAVES = NT / 64;
    const int tid = threadIdx.x, wave = tid >> 6;
    sh.best[tid] = best;
    if (tid == 0) { sh.n_threads = 0; sh.n_cand = 0; }
    __syncthreads();
    int rank = 0;
#pragma unroll 8
    for (int u = 0; u < 64; ++u) rank += sh.best[wave * 64 + u] > best;
    // equal keys are all 0: then the bound is 0 if the rank lies among them
    const int want = (top + WAVES - 1) / WAVES - 1;
    const uint64_t hit = __ballot(rank == want);
    if (hit == 0) {
        if ((tid & 63) == 0) sh.least[wave] = 0;
    } else if (rank == want) {
        sh.least[wave] = best;
    }
    __syncthreads();
    uint64_t t = sh.least[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t = min(t, sh.least[w]);
    if (best != 0 && best >= t) sh.threads[atomicAdd(&sh.n_threads, 1)] = tid;
    __syncthreads();
    return t;
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

template <int NT> __device__ inline void add_candidate(TopShared<NT> &sh, uint64_t key)
{
    const int at = atomicAdd(&sh.n_cand, 1);
    if (at < kCandidates) sh.cand[at] = key;
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
        __syncthreads();                       // all have read it before it changes
        const bool fits = n <= kCandidates;
        if (fits) { at += width; have = n; }
        else width = kNarrow;                  // and this step again
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
    rank_candidates(sh, have, top, emit);
}

// ------------------------------------------------------------------ joining lanes -------
template <int NT> struct StatsShared {
    float m[NT / 64], s[NT / 64], d[NT / 64];
};

// A lane's value from the lane CTRL says, inside rows of 16.
template <int CTRL> __device__ inline float dpp(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                                 0xf, 0xf, true));
}
template <int CTRL> __device__ inline void join_dpp(RowStats &st)
{
    st.join(dpp<CTRL>(st.m), dpp<CTRL>(st.s), dpp<CTRL>(st.d));
}

// Every thread gets the workgroup's joined sums (in the same order each time). Lanes are
// joined by cross-lane moves up to 16, then by shuffles.
template <int NT> __device__ inline RowStats join_stats(StatsShared<NT> &sh, RowStats st)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    join_dpp<0xb1>(st);          // lane ^ 1
    join_dpp<0x4e>(st);          // lane ^ 2
    join_dpp<0x141>(st);         // mirrored in 8 lanes: the other four
    join_dpp<0x140>(st);         // mirrored in 16: the other eight
    st.join(__shfl_xor(st.m, 16), __shfl_xor(st.s, 16), __shfl_xor(st.d, 16));
    st.join(__shfl_xor(st.m, 32), __shfl_xor(st.s, 32), __shfl_xor(st.d, 32));
    if (lane == 0) { sh.m[wave] = st.m; sh.s[wave] = st.s; sh.d[wave] = st.d; }
    __syncthreads();
    RowStats all;
    for (int w = 0; w < NT / 64; ++w) all.join(sh.m[w], sh.s[w], sh.d[w]);
    return all;
}

struct RowResult {
    float lse, entropy;
};
__device__ inline RowResult row_result(const RowStats &st)
{
    if (st.s == 0.0f) return {kNegInf, 0.0f};            // nothing but -infinity
    const float logs = __builtin_logf(st.s);
    return {st.m + logs, logs - kLn2 * (st.d / st.s)};
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
    const RowResult r = row_result(st);
    // x - m is small where x is likely, so it is taken before log s is
    float lp = (token.x - st.m) - __builtin_logf(st.s);
    if (st.s == 0.0f) lp = kNegInf;
    if (token.t >= p.V) lp = __builtin_nanf("");
    p.logprobs[row] = token.t < 0 ? 0.0f : lp;
    if (p.entropy) p.entropy[row] = r.entropy;
    if (p.lse) p.lse[row] = r.lse;
}
__device__ inline void write_top(const RowArgs &p, int64_t row, const RowStats &st, int r,
                                 uint64_t key)
{
    const float x = key_value(key);
    p.top_logprobs[row * p.top + r] =
        st.s == 0.0f ? (x == x ? kNegInf : x) : (x - st.m) - __builtin_logf(st.s);
    p.top_tokens[row * p.top + r] = key_index(key);
}

// ------------------------------------------------------------------ the pass ------------
// One workgroup per (row, part). A thread's elements: up to one of the head before the
// first 16-byte boundary, then the chunks tid, tid + 256, ... of 16 bytes, then up to one
// of the tail. U chunks are in flight, and the peak is raised once for them. HBM-bound where rows fill the card; the
// arithmetic (a conversion, 1/2 max, a difference, a product, an exponential at a quarter of
// the rate, a max, two sums an element) comes to most of that time.
template <int DT, bool TOP, int NT, int U>
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
    if (p.splits == 1 && tid == 0) token = load_token<DT>(p, row);

    RowStats st;
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
    auto take1 = [&](int at) __attribute__((always_inline)) {
        const float v = Elem<DT>::widen(x[at]);
        note(v, at);
        st.raise(v);
        st.add(v);
    };
    if (tid < head) take1(tid);
    auto load = [&](Pack<T, W> (&b)[U], int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            b[u] = load_pack<T, W>(body + int64_t(min(c + u * NT, chunks - 1)) * W);
    };
    auto widen = [&](float (&v)[W], const Pack<T, W> &b, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = Elem<DT>::widen(b.v[j]);
        float peak = v[0];
#pragma unroll
        for (int j = 1; j < W; ++j) peak = __builtin_fmaxf(peak, v[j]);
        note(peak, head + c * W);
        return peak;
    };
    int c = tid;
    for (; c + (U - 1) * NT < chunks; c += U * NT) {
        Pack<T, W> b[U];
        float v[U][W], peak = kNegInf;
        load(b, c);
#pragma unroll
        for (int u = 0; u < U; ++u) peak = __builtin_fmaxf(peak, widen(v[u], b[u], c + u * NT));
        st.raise(peak);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j) st.add(v[u][j]);
    }
    if (c < chunks) {                                     // fewer than U are left
        Pack<T, W> b[U];
        load(b, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u * NT >= chunks) break;
            float v[W];
            st.raise(widen(v, b[u], c + u * NT));
#pragma unroll
            for (int j = 0; j < W; ++j) st.add(v[j]);
        }
    }
    if (tid < n - tail) take1(tail + tid);

    const RowStats all = join_stats(stats, st);
    RowPart *out = reinterpret_cast<RowPart *>(p.parts + int64_t(blockIdx.x) * p.part_bytes);
    if (tid == 0) {
        if (p.splits == 1) write_row(p, row, all, token);
        else *out = RowPart{all.m, all.s, all.d, 0.0f};
    }
    if constexpr (TOP) {
        const uint64_t mine = empty ? 0 : uint64_t(best) << 32 | (0xffffffffu - uint32_t(best_at));
        uint64_t floor = top_bound(tops, mine, p.top);
        // T's group reaches W - 1 elements behind its first
        const uint32_t low = uint32_t(floor);
        floor -= min(low, uint32_t(W - 1));
        // the threads' chunks, and one more slot for their head and tail
        const int per = (chunks + NT - 1) / NT + 1;
        auto look = [&](int slot, uint64_t least) {
            const int u = tops.threads[slot / per], i = slot % per;
            auto offer = [&](float v, int at) {
                const uint64_t k = key_of(v, uint32_t(at));
                if (k >= least) add_candidate(tops, k);
            };
            if (i == per - 1) {
                if (u < head) offer(Elem<DT>::widen(x[u]), u);
                if (u < n - tail) offer(Elem<DT>::widen(x[tail + u]), tail + u);
                return;
            }
            const int chunk = u + i * NT;
            if (chunk >= chunks) return;
            const Pack<T, W> b = load_pack<T, W>(body + int64_t(chunk) * W);
#pragma unroll
            for (int j = 0; j < W; ++j) offer(Elem<DT>::widen(b.v[j]), head + chunk * W + j);
        };
        const int slots = tops.n_threads * per;
        if (p.splits > 1) {
            uint64_t *keys = reinterpret_cast<uint64_t *>(out + 1);
            // a part shorter than `top` leaves its last keys empty
            if (tid < p.top && tid >= n) keys[tid] = 0;
            // indices in the row
            select_top(tops, floor, slots, p.top, look,
                       [&](int r, uint64_t k) { keys[r] = k - uint32_t(first); });
        } else {
            select_top(tops, floor, slots, p.top, look,
                       [&](int r, uint64_t k) { write_top(p, row, all, r, k); });
        }
    }
}

// Joins a row's parts: the sums in one order of the parts, the alternatives from the parts'
// lists (in the parts' order, so every key is a group of its own).
template <int DT, bool TOP>
__global__ __launch_bounds__(256) void k_row_join(RowArgs p)
{
    constexpr int NT = 256;
    __shared__ StatsShared<NT> stats;
    __shared__ TopShared<TOP ? NT : 64> tops;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const char *parts = p.parts + row * p.splits * p.part_bytes;
    RowToken token{};
    if (tid == 0) token = load_token<DT>(p, row);
    const int n = TOP ? p.splits * p.top : 0;
    auto key_at = [&](int i) {
        const int s = i / p.top;
        return reinterpret_cast<const uint64_t *>(parts + s * p.part_bytes +
                                                  sizeof(RowPart))[i - s * p.top];
    };
    uint64_t best = 0;
    for (int i = tid; i < n; i += NT) best = max(best, key_at(i));
    RowStats st;
    for (int s = tid; s < p.splits; s += NT) {
        const RowPart *q = reinterpret_cast<const RowPart *>(parts + s * p.part_bytes);
        st.join(q->peak, q->sum, q->dot);
    }
    const RowStats all = join_stats(stats, st);
    if (tid == 0) write_row(p, row, all, token);
    if constexpr (TOP) {
        const uint64_t floor = max(top_bound(tops, best, p.top), uint64_t(1));
        select_top(tops, floor, n, p.top,
                   [&](int slot, uint64_t least) {
                       const uint64_t k = key_at(slot);
                       if (k >= least) add_candidate(tops, k);
                   },
                   [&](int r, uint64_t k) { write_top(p, row, all, r, k); });
    }
}

// ------------------------------------------------------------------ the gradient --------
struct GradArgs {
    const void *logits;
    void *grad;
    const void *tokens;
    const float *lse, *entropy, *g_logprob, *g_entropy, *g_lse;
    int64_t ld, ldg;
    int M, V, token_bytes, parts, part_len;
};

// One workgroup per (row, part): dx = -p (a + h (logp + H)), plus g at the token, with
// a = g - g_lse and h = g_entropy.
constexpr int kGradThreads = 256;
template <int DT>
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
    float g = p.g_logprob && t >= 0 ? p.g_logprob[row] : 0.0f;
    float h = p.g_entropy ? p.g_entropy[row] : 0.0f;
    const float entropy = p.g_entropy ? p.entropy[row] : 0.0f;
    float a = g - (p.g_lse ? p.g_lse[row] : 0.0f);
    if (t >= p.V && p.g_logprob) a = __builtin_nanf("");
    if (lse == kNegInf) { lse = 0.0f; g = 0.0f; a = 0.0f; h = 0.0f; }   // p = 0 throughout
    const int64_t at = t - first;                         // the token's element of the part
    auto value = [&](float v, bool is_token) __attribute__((always_inline)) {
        const float logp = v - lse;
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
        const Pack<T, W> in = load_pack<T, W>(x + e);
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
        store_pack(out + e, o);
    }
}

}  // namespace sgemm
