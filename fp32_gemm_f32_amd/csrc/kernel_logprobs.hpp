// kernel_logprobs.hpp -- kernels of token_logprobs.h: one pass over each row of logits for
// its log-sum-exp, entropy and top alternatives, the join of rows that were split, and the
// gradient.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_common.hpp"

namespace sgemm {

constexpr int kRowThreads = 256;          // threads of a workgroup on one row or part
constexpr int kRowWaves = kRowThreads / 64;
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

__device__ inline uint64_t lane_key(uint64_t key, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(key), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(key >> 32), lane);
    return uint64_t(hi) << 32 | lo;
}

// A wave's list of its `top` largest keys so far: lane j holds the j-th largest, 0 where
// there is none yet.
struct WaveList {
    uint64_t key = 0, least = 0;      // least: the list's last key (uniform)

    // one candidate per lane (0: none)
    __device__ void insert(uint64_t candidate, int top)
    {
        const int lane = threadIdx.x & 63;
        uint64_t todo = __ballot(candidate > least);
        while (todo != 0) {
            const int from = __builtin_ctzll(todo);
            todo &= todo - 1;
            const uint64_t k = lane_key(candidate, from);
            if (k <= least) continue;
            const int at = __builtin_popcountll(__ballot(key > k));
            const uint64_t up = __shfl_up(key, 1);
            key = lane < at ? key : lane == at ? k : up;
            least = lane_key(key, top - 1);
        }
    }
};

struct TopShared {
    float best[kRowThreads];
    uint64_t lists[kRowWaves][64];
    float bound;
};

// The `top` largest of the elements that the workgroup's threads hold, given each thread's
// own best. A first bound is the top-th largest of the threads' bests: at least `top`
// elements reach it, and only the threads whose best does can hold one. Their elements are
// looked at again, a wave at a time, and those that reach the bound go through the wave's
// sorted list; then the waves' lists are ranked against each other. With values in no
// order about `top` of the 256 threads are looked at again. Ties and sorted rows bring
// more, at worst all.
//   again(u, i): the key of element i of thread u, 0 past its last
//   count(u):    how many elements thread u holds
//   emit(r, k):  takes the key of rank r < top
template <typename Again, typename Count, typename Emit>
__device__ inline void select_top(TopShared &sh, float best, int top, Again again, Count count,
                                  Emit emit)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    best += 0.0f;                              // -0 ranks as 0
    sh.best[tid] = best;
    __syncthreads();
    int rank = 0;
    for (int u = 0; u < kRowThreads; ++u) {
        const float x = sh.best[u];
        rank += x > best || (x == best && u < tid);
    }
    if (rank == top - 1) sh.bound = best;
    __syncthreads();
    const float bound = sh.bound;
    const uint32_t floor = bound == kNegInf ? 0u : ordered(bound);
    WaveList list;
    int turn = 0;
    for (int g = 0; g < kRowThreads; g += 64) {
        // the threads to look at again take turns over the waves
        uint64_t mine = __ballot(sh.best[g + lane] >= bound);
        while (mine != 0) {
            const int u = g + __builtin_ctzll(mine);
            mine &= mine - 1;
            if (turn++ % kRowWaves != wave) continue;
            const int n = count(u);
            for (int i = 0; i < n; i += 64) {
                uint64_t k = again(u, i + lane);
                if (uint32_t(k >> 32) < floor) k = 0;
                list.insert(k, top);
            }
        }
    }
    sh.lists[wave][lane] = lane < top ? list.key : 0;
    __syncthreads();
    if (lane < top && list.key != 0) {
        int r = 0;
        for (int w = 0; w < kRowWaves; ++w)
            for (int j = 0; j < top; ++j) r += sh.lists[w][j] > list.key;
        if (r < top) emit(r, list.key);
    }
}

// ------------------------------------------------------------------ joining lanes -------
struct StatsShared {
    float m[kRowWaves], s[kRowWaves], d[kRowWaves];
};

// Every thread gets the workgroup's joined sums (in the same order each time).
__device__ inline RowStats join_stats(StatsShared &sh, RowStats st)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1)
        st.join(__shfl_xor(st.m, x), __shfl_xor(st.s, x), __shfl_xor(st.d, x));
    if (lane == 0) { sh.m[wave] = st.m; sh.s[wave] = st.s; sh.d[wave] = st.d; }
    __syncthreads();
    RowStats all;
    for (int w = 0; w < kRowWaves; ++w) all.join(sh.m[w], sh.s[w], sh.d[w]);
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

// The log-probability of the row's token (the edge rules of token_logprobs.h).
template <int DT>
__device__ inline float token_logprob(const RowArgs &p, int64_t row, const RowStats &st)
{
    const int64_t t = token_of(p.tokens, p.token_bytes, row);
    if (t < 0) return 0.0f;
    if (t >= p.V) return __builtin_nanf("");
    if (st.s == 0.0f) return kNegInf;
    typedef typename Elem<DT>::type T;
    const float x = Elem<DT>::widen(static_cast<const T *>(p.logits)[row * p.ld + t]);
    // x - m is small where x is likely, so it is taken before log s is
    return (x - st.m) - __builtin_logf(st.s);
}

template <int DT>
__device__ inline void write_row(const RowArgs &p, int64_t row, const RowStats &st)
{
    if (threadIdx.x == 0) {
        const RowResult r = row_result(st);
        p.logprobs[row] = token_logprob<DT>(p, row, st);
        if (p.entropy) p.entropy[row] = r.entropy;
        if (p.lse) p.lse[row] = r.lse;
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

// ------------------------------------------------------------------ the pass ------------
// One workgroup per (row, part). A thread's elements: up to one of the head before the
// first 16-byte boundary, then the chunks tid, tid + 256, ... of 16 bytes, then up to one
// of the tail.
template <int DT, bool TOP>
__global__ __launch_bounds__(kRowThreads) void k_row_pass(RowArgs p)
{
    typedef typename Elem<DT>::type T;
    constexpr int W = 16 / sizeof(T);
    constexpr int U = 4;                                  // chunks in flight per thread
    __shared__ StatsShared stats;
    __shared__ TopShared tops[TOP ? 1 : 1];
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

    RowStats st;
    float best = kNegInf;
    auto take1 = [&](float v) __attribute__((always_inline)) {
        best = __builtin_fmaxf(best, v);
        st.raise(v);
        st.add(v);
    };
    if (tid < head) take1(Elem<DT>::widen(x[tid]));
    if (tid < n - tail) take1(Elem<DT>::widen(x[tail + tid]));
    auto take = [&](const Pack<T, W> &c) __attribute__((always_inline)) {
        float v[W], peak;
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = Elem<DT>::widen(c.v[j]);
        peak = v[0];
#pragma unroll
        for (int j = 1; j < W; ++j) peak = __builtin_fmaxf(peak, v[j]);
        best = __builtin_fmaxf(best, peak);
        st.raise(peak);
#pragma unroll
        for (int j = 0; j < W; ++j) st.add(v[j]);
    };
    int c = tid;
    for (; c + (U - 1) * kRowThreads < chunks; c += U * kRowThreads) {
        Pack<T, W> b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) b[u] = load_pack<T, W>(body + int64_t(c + u * kRowThreads) * W);
#pragma unroll
        for (int u = 0; u < U; ++u) take(b[u]);
    }
    for (; c < chunks; c += kRowThreads) take(load_pack<T, W>(body + int64_t(c) * W));

    const RowStats all = join_stats(stats, st);
    RowPart *out = reinterpret_cast<RowPart *>(p.parts + int64_t(blockIdx.x) * p.part_bytes);
    if (p.splits == 1) write_row<DT>(p, row, all);
    else if (tid == 0) *out = RowPart{all.m, all.s, all.d, 0.0f};
    if constexpr (TOP) {
        auto count = [&](int u) {
            const int mine = u < chunks ? (chunks - u + kRowThreads - 1) / kRowThreads : 0;
            return mine * W + 2;
        };
        auto again = [&](int u, int i) -> uint64_t {
            int e;                                        // element of the part
            if (i == 0) e = u < head ? u : -1;
            else if (i == 1) e = u < n - tail ? tail + u : -1;
            else {
                const int chunk = u + (i - 2) / W * kRowThreads;
                e = chunk < chunks ? head + chunk * W + (i - 2) % W : -1;
            }
            return e < 0 ? 0 : key_of(Elem<DT>::widen(x[e]), uint32_t(first + e));
        };
        if (p.splits > 1) {
            uint64_t *keys = reinterpret_cast<uint64_t *>(out + 1);
            // a part shorter than `top` leaves its last keys empty
            if (tid < p.top && tid >= n) keys[tid] = 0;
            select_top(tops[0], best, p.top, again, count,
                       [&](int r, uint64_t k) { keys[r] = k; });
        } else {
            select_top(tops[0], best, p.top, again, count,
                       [&](int r, uint64_t k) { write_top(p, row, all, r, k); });
        }
    }
}

// Joins a row's parts: the sums in the parts' order, the alternatives from the parts' lists.
template <int DT, bool TOP>
__global__ __launch_bounds__(kRowThreads) void k_row_join(RowArgs p)
{
    __shared__ TopShared tops[1];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const char *parts = p.parts + row * p.splits * p.part_bytes;
    RowStats all;
    for (int s = 0; s < p.splits; ++s) {
        const RowPart *q = reinterpret_cast<const RowPart *>(parts + s * p.part_bytes);
        all.join(q->peak, q->sum, q->dot);
    }
    write_row<DT>(p, row, all);
    if constexpr (TOP) {
        const int n = p.splits * p.top;
        auto key_at = [&](int i) {
            const int s = i / p.top;
            return reinterpret_cast<const uint64_t *>(parts + s * p.part_bytes +
                                                      sizeof(RowPart))[i - s * p.top];
        };
        float best = kNegInf;
        for (int i = tid; i < n; i += kRowThreads) {
            const uint64_t k = key_at(i);
            const float v = k == 0 ? kNegInf : key_value(k);
            best = __builtin_fmaxf(best, v);
        }
        select_top(tops[0], best, p.top,
                   [&](int u, int i) -> uint64_t {
                       const int at = u + i * kRowThreads;
                       return at < n ? key_at(at) : 0;
                   },
                   [&](int u) { return u < n ? (n - u + kRowThreads - 1) / kRowThreads : 0; },
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
template <int DT>
__global__ __launch_bounds__(kRowThreads) void k_row_gradient(GradArgs p)
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
    const float shift = entropy;
    auto value = [&](float v, int64_t e) __attribute__((always_inline)) {
        const float logp = v - lse;
        const float pr = __builtin_amdgcn_exp2f(logp * kLog2e);
        const float w = __builtin_fmaf(h, __builtin_fmaxf(logp, -1000.0f) + shift, a);
        const float dx = -pr * w;
        return e == at ? dx + g : dx;
    };
    const int head = min(n, int((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
    const int chunks = (n - head) / W;
    const int tail = head + chunks * W;
    if (tid < head) out[tid] = Elem<DT>::narrow(value(Elem<DT>::widen(x[tid]), tid));
    if (tid < n - tail)
        out[tail + tid] = Elem<DT>::narrow(value(Elem<DT>::widen(x[tail + tid]), tail + tid));
    for (int c = tid; c < chunks; c += kRowThreads) {
        const int64_t e = head + int64_t(c) * W;
        const Pack<T, W> in = load_pack<T, W>(x + e);
        Pack<T, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) o.v[j] = Elem<DT>::narrow(value(Elem<DT>::widen(in.v[j]), e + j));
        store_pack(out + e, o);
    }
}

}  // namespace sgemm
