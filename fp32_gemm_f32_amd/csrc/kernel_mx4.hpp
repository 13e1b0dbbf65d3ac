// kernel_mx4.hpp -- kernels of gemm_mx4.h: the quantiser to microscaled 4-bit elements, its inverse,
// and what the kernels of the product share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "byte_tiles.hpp"
#include "ops_common.hpp"

namespace sgemm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ elements -----------
// 2^(byte - 127) as FP32 (0 is the denormal 2^-127).
__device__ inline float mx4_unit(uint32_t byte)
{
    return byte == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
}
// The scale's byte of a block whose largest magnitude has these bits as FP32: its exponent less the
// format's own largest (2), 255 where it is no number. (A denormal's exponent reads as 0.)
__device__ inline uint32_t mx4_scale(uint32_t peak)
{
    const int e = int(peak >> 23);
    return e == 255 ? 255u : uint32_t(max(e - 2, 0));
}

// 8 elements over `unit` as codes, the first in the lowest bits: gfx950's conversion rounds to
// nearest even and saturates, for every value and power of two.
template <typename T> __device__ inline uint32_t mx4_encode(const Pack<T, 8> &x, float unit)
{
    uint32_t q = 0;
    const auto pair = [&](auto i) __attribute__((always_inline)) {
        constexpr int e = 2 * decltype(i)::value;
        if constexpr (sizeof(T) == 4) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x.v[e], x.v[e + 1], unit, e / 2);
        } else if constexpr (__is_same(T, __bf16)) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16x2{x.v[e], x.v[e + 1]}, unit, e / 2);
        } else {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, f16x2{x.v[e], x.v[e + 1]}, unit, e / 2);
        }
    };
    static_for<0, 4>(pair);
    return q;
}
template <typename T> __device__ inline Pack<T, 8> mx4_decode(uint32_t q, float unit)
{
    Pack<T, 8> x;
    static_for<0, 4>([&](auto i) __attribute__((always_inline)) {
        constexpr int e = 2 * decltype(i)::value;
        if constexpr (sizeof(T) == 4) {
            const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, unit, e / 2);
            x.v[e] = v[0];
            x.v[e + 1] = v[1];
        } else if constexpr (__is_same(T, __bf16)) {
            const auto v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, e / 2);
            x.v[e] = v[0];
            x.v[e + 1] = v[1];
        } else {
            const auto v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, e / 2);
            x.v[e] = v[0];
            x.v[e + 1] = v[1];
        }
    });
    return x;
}

struct Mx4RowArgs {
    const void *X;             // (the inverse: the values written)
    int64_t ldx;
    uint8_t *Q;
    int64_t ldq;
    uint8_t *scales;
    int64_t lds;
    int M, K, units;           // units of 8 elements to a row, whole blocks of them
    Divisor by_units;
};

// Bytes that what is left of a row takes. A row is filled up to whole blocks of four units, so a unit may
// start behind its end: `left` is below 0 then, and -1 / 2 is 0.
constexpr int mx4_bytes_of(int left) { return left <= 0 ? 0 : left / 2 + left % 2; }
static_assert(mx4_bytes_of(-1) == 0 && mx4_bytes_of(-25) == 0 && mx4_bytes_of(0) == 0 && mx4_bytes_of(1) == 1 &&
              mx4_bytes_of(7) == 4 && mx4_bytes_of(8) == 4 && mx4_bytes_of(0x7fffffff) == 0x40000000, "a row's end");

// 8 elements; STREAM: read past the caches.
template <bool STREAM, typename T> __device__ inline Pack<T, 8> mx4_load_unit(const T *x)
{
    if constexpr (!STREAM) {
        return load_pack<T, 8>(x);
    } else if constexpr (sizeof(T) == 2) {
        return load_pack_stream<T, 8>(x);
    } else {
        struct { Pack<T, 4> half[2]; } v = {{load_pack_stream<T, 4>(x), load_pack_stream<T, 4>(x + 4)}};
        return __builtin_bit_cast(Pack<T, 8>, v);
    }
}

// Four lanes share a block, 8 elements each; U times 256 lanes to a workgroup, their loads first.
// HBM-bound: 2 or 4 bytes in and 17 / 32 out of an element. 8192 x 8192 bf16 28.6 us (5.9 TB/s); loads past
// the caches against loads that stay there, taken in turn: 27.8 and 28.4, at 16384 x 8192 53.2 and 60.3.
template <int DT, int U>
__global__ __launch_bounds__(256) void k_mx4_quantize(Mx4RowArgs p)
{
    typedef typename Elem<DT>::type T;
    Pack<T, 8> v[U];
    int row[U], unit[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e = (int(blockIdx.x) * U + u) * 256 + int(threadIdx.x);
        row[u] = divide(e, p.by_units);
        unit[u] = e - row[u] * p.units;
        const int k = unit[u] * 8;
        const T *x = static_cast<const T *>(p.X) + row[u] * p.ldx + k;
        const bool mine = row[u] < p.M;
        const int left = p.K - k;                         // (k + 8 may pass 31 bits)
        if (mine && left >= 8) {
            v[u] = mx4_load_unit<U != 1>(x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[u].v[j] = mine && j < left ? x[j] : T(0.0f);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t peak = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            peak = max(peak, __builtin_bit_cast(uint32_t, Elem<DT>::widen(v[u].v[j])) & 0x7fffffffu);
        const auto moved = [](uint32_t a, auto ctrl) {
            return uint32_t(__builtin_amdgcn_update_dpp(0, int(a), decltype(ctrl)::value, 0xf, 0xf, true));
        };
        peak = max(peak, moved(peak, std::integral_constant<int, 0xb1>{}));     // lane ^ 1
        peak = max(peak, moved(peak, std::integral_constant<int, 0x4e>{}));     // lane ^ 2
        const uint32_t s = mx4_scale(peak);
        const uint32_t q = s == 255 ? 0 : mx4_encode<T>(v[u], mx4_unit(s));
        if (row[u] >= p.M) continue;
        const int k = unit[u] * 8;
        uint8_t *out = p.Q + row[u] * p.ldq + k / 2;
        const int bytes = mx4_bytes_of(p.K - k);
        if (bytes >= 4) {
            *reinterpret_cast<Pack<uint32_t, 1> *>(out) = Pack<uint32_t, 1>{{q}};
        } else {
            for (int j = 0; j < bytes; ++j) out[j] = uint8_t(q >> 8 * j);
        }
        if (unit[u] % 4 == 0 && k < p.K) p.scales[row[u] * p.lds + unit[u] / 4] = uint8_t(s);
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_mx4_dequantize(Mx4RowArgs p)
{
    typedef typename Elem<DT>::type T;
    const int e = int(blockIdx.x) * 256 + int(threadIdx.x);
    const int row = divide(e, p.by_units), unit = e - row * p.units, k = unit * 8;
    if (row >= p.M || k >= p.K) return;
    const uint8_t *in = p.Q + row * p.ldq + k / 2;
    const float size = mx4_unit(p.scales[row * p.lds + unit / 4]);
    T *y = static_cast<T *>(const_cast<void *>(p.X)) + row * p.ldx + k;
    const int left = p.K - k;                             // (k + 8 may pass 31 bits)
    if (left >= 8) {
        store_pack(y, mx4_decode<T>(load_pack<uint32_t, 1>(reinterpret_cast<const uint32_t *>(in)).v[0], size));
        store_data_guard<true>();                         // the other branch begins with writes of its registers
    } else {
        uint32_t q = 0;
        for (int j = 0; j < (left + 1) / 2; ++j) q |= uint32_t(in[j]) << 8 * j;
        const Pack<T, 8> v = mx4_decode<T>(q, size);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) y[j] = v.v[j];
    }
}

// ------------------------------------------------------------------ the product ---------
struct Mx4Args {
    const uint8_t *A, *B, *sa, *sb;
    const float *bias;         // or NULL
    void *C;
    float *partial;            // splits > 1: sums of split s at partial + s * M * N
    int64_t lda, ldb, ldsa, ldsb, ldc;
    int64_t sa_bytes, sb_bytes;// tiles: all of the scales'
    int sa_step, sb_step;      // tiles: from the 16 scales of a row for two panels to the next 16
    int M, N, KB;              // KB: bytes to a row, K / 2
    int c_dtype, tiles_m, tiles_n;
    uint32_t group_mul;        // division by kGroupM * tiles_n without dividing: see tile_of
    int group_shift;
    bool stream;               // C's rows start on lines of 64 bytes: store past the caches
    int splits, chunk;         // split s covers bytes [s * chunk, min(KB, (s + 1) * chunk))
};

__device__ inline void mx4_store_one(int dtype, void *C, int64_t at, float x)
{
    const float v[1] = {x};
    store_values_as<1>(dtype, C, at, v, 1);
}

__device__ inline i32x4 mx4_load_tail(const uint8_t *row, int k, int kn)
{
    return load_tail(reinterpret_cast<const int8_t *>(row), k, kn);
}
__device__ inline i32x4 mx4_load16(const uint8_t *p)
{
    return __builtin_bit_cast(i32x4, load_pack<int, 4>(reinterpret_cast<const int *>(p)));
}

// Adds the splits' sums in their order; one thread per element of C, strided over the grid.
__global__ __launch_bounds__(256) void k_mx4_join(Mx4Args p)
{
    const int64_t total = int64_t(p.M) * p.N;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < total; e += int64_t(gridDim.x) * 256) {
        const int64_t m = e / p.N;
        const int n = int(e - m * p.N);
        float sum = 0.0f;
        for (int s = 0; s < p.splits; ++s) sum += p.partial[s * total + e];
        mx4_store_one(p.c_dtype, p.C, m * p.ldc + n, p.bias ? sum + p.bias[n] : sum);
    }
}

// What is put in place first, in one launch, for a launch of its own costs 2.5 us: rows of A and of B in
// whole chunks, and scales in another order, 16 of a row (a group, two panels' worth) at (group rows + row)
// 16 with zeros behind the last. Of those a wave takes 16 rows and four groups: it reads 64 bytes of
// each row and writes four times 256.
struct Mx4Scales {
    const uint8_t *src;
    uint8_t *dst;
    int64_t ld;
    int rows, blocks;          // workgroups, 64 rows and four groups each
    int across;                // of them to 64 rows
};
struct Mx4Place {
    Rows16 rows[2];
    Mx4Scales scales[2];
    int bytes, count;          // of a row's elements; scales to a row
};
__device__ inline void mx4_arrange(const Mx4Scales &p, int block, int scales)
{
    const int down = block / p.across;
    const int row = down * 64 + int(threadIdx.x >> 6) * 16 + int(threadIdx.x & 15);
    const int group = (block - down * p.across) * 4 + int(threadIdx.x >> 4 & 3);
    if (row >= p.rows || group * 16 >= scales) return;
    const uint8_t *from = p.src + row * p.ld;
    const i32x4 v = group * 16 + 16 <= scales ? mx4_load16(from + group * 16) : mx4_load_tail(from, group * 16, scales);
    *reinterpret_cast<i32x4 *>(p.dst + (int64_t(group) * p.rows + row) * 16) = v;
}
__global__ __launch_bounds__(256) void k_mx4_place(Mx4Place p)
{
    int block = blockIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (block >= 0 && block < p.rows[i].blocks) put_rows_in_place(p.rows[i], block, p.bytes);
        block -= p.rows[i].blocks;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (block >= 0 && block < p.scales[i].blocks) mx4_arrange(p.scales[i], block, p.count);
        block -= p.scales[i].blocks;
    }
}

// K == 0: the empty sum plus the bias.
__global__ __launch_bounds__(256) void k_mx4_empty(Mx4Args p)
{
    const int64_t total = int64_t(p.M) * p.N;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < total; e += int64_t(gridDim.x) * 256) {
        const int64_t m = e / p.N;
        const int n = int(e - m * p.N);
        mx4_store_one(p.c_dtype, p.C, m * p.ldc + n, p.bias ? p.bias[n] : 0.0f);
    }
}

}  // namespace sgemm
