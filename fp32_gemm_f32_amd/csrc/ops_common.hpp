// ops_common.hpp -- what the units of the 8-bit product (gemm_i8.hip) and of the token
// log-probabilities (token_logprobs.hip) share: launching, the device's compute units,
// region checks in bytes, and loads and stores of the three element types.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "sgemm_dtype.h"
#include "sgemm_f32.h"

namespace sgemm {
namespace {

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, void *stream, Args... args)
{
    static_assert(sizeof...(KArgs) == sizeof...(Args), "argument count");
    void *argv[] = {static_cast<void *>(&args)...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kern), grid, block,
                                         argv, 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SGEMM_OK : SGEMM_ELAUNCH;
}

// The most workgroups one launch may have: HIP takes fewer than 2^32 work items in a dimension. What
// needs more goes out in several launches, each over its own rows or columns.
inline int64_t most_groups(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

// Compute units of the current device, looked up once per device.
inline int device_cus(int *out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return SGEMM_ELAUNCH;
    if (dev >= 0 && dev < 64) {
        const int c = known[dev].load(std::memory_order_relaxed);
        if (c > 0) { *out = c; return SGEMM_OK; }
    }
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
        return SGEMM_ELAUNCH;
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    *out = n;
    return SGEMM_OK;
}

inline bool known_dtype(int t)
{
    return t == SGEMM_DTYPE_F32 || t == SGEMM_DTYPE_BF16 || t == SGEMM_DTYPE_F16;
}
inline int dtype_bytes(int t) { return t == SGEMM_DTYPE_F32 ? 4 : 2; }

// A region in bytes: rows of `cols` elements of `size` bytes, `ld` elements apart. The
// products saturate, so that no leading dimension wraps a comparison.
struct Region {
    const void *p;
    uint64_t bytes;
};
inline Region region(const void *p, int64_t rows, int64_t cols, int64_t ld, int size)
{
    if (rows <= 0 || cols <= 0) return {p, 0};
    const __int128 n = (static_cast<__int128>(rows - 1) * ld + cols) * size;
    const __int128 most = static_cast<__int128>(1) << 62;
    return {p, static_cast<uint64_t>(n < most ? n : most)};
}
inline bool bad_region(const Region &r, int align)
{
    if (r.bytes == 0) return false;
    return r.p == nullptr || reinterpret_cast<uintptr_t>(r.p) % align != 0;
}
inline bool overlaps(const Region &a, const Region &b)
{
    if (a.bytes == 0 || b.bytes == 0 || a.p == nullptr || b.p == nullptr) return false;
    const uint64_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 ? b0 - a0 < a.bytes : a0 - b0 < b.bytes;
}

// ---------------------------------------------------------------- elements on the GPU ---

template <int DT> struct Elem;
template <> struct Elem<SGEMM_DTYPE_F32> {
    typedef float type;
    __device__ static float widen(float x) { return x; }
    __device__ static float narrow(float x) { return x; }
};
template <> struct Elem<SGEMM_DTYPE_BF16> {
    typedef __bf16 type;
    __device__ static float widen(__bf16 x) { return static_cast<float>(x); }
    __device__ static __bf16 narrow(float x) { return static_cast<__bf16>(x); }
};
template <> struct Elem<SGEMM_DTYPE_F16> {
    typedef _Float16 type;
    __device__ static float widen(_Float16 x) { return static_cast<float>(x); }
    // x is rounded to FP32 before, and to FP16 here. The empty asm keeps the two apart: the compiler
    // otherwise makes one v_fma_mixlo_f16 of a multiply-add and this, which rounds once, in some
    // kernels (and for some elements) and not in others.
    __device__ static _Float16 narrow(float x)
    {
        asm("" : "+v"(x));
        return static_cast<_Float16>(x);
    }
};

// W consecutive elements at an address aligned to one element only: the compiler makes one
// load or store of it, which gfx950 serves at any alignment (and at full speed where the
// address is a multiple of the whole).
template <typename T, int W> struct __attribute__((packed)) Pack {
    T v[W];
};
template <typename T, int W> __device__ inline Pack<T, W> load_pack(const T *p)
{
    return *reinterpret_cast<const Pack<T, W> *>(p);
}
// The same with the hint that the line is not used again soon.
template <int BYTES> struct Bits;
template <> struct Bits<2> { typedef uint16_t type; };
template <> struct Bits<4> { typedef uint32_t type; };
template <> struct Bits<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Bits<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <typename T, int W> __device__ inline Pack<T, W> load_pack_stream(const T *p)
{
    typedef typename Bits<sizeof(T) * W>::type B;
    typedef B __attribute__((aligned(alignof(T)))) unaligned;
    return __builtin_bit_cast(Pack<T, W>, static_cast<B>(__builtin_nontemporal_load(reinterpret_cast<const unaligned *>(p))));
}
// Results leave this way where whole lines do: they are written once, and the caches serve the
// operands instead (gradient of 511 x 32001 f32 27.4 to 22.3 us, quantiser of 8192 x 4000 bf16 20.9 to
// 17.4).
template <typename T, int W> __device__ inline void store_pack_stream(T *p, const Pack<T, W> &x)
{
    typedef typename Bits<sizeof(T) * W>::type B;
    typedef B __attribute__((aligned(alignof(T)))) unaligned;
    __builtin_nontemporal_store(__builtin_bit_cast(B, x), reinterpret_cast<unaligned *>(p));
}
template <typename T, int W> __device__ inline void store_pack(T *p, const Pack<T, W> &x)
{
    *reinterpret_cast<Pack<T, W> *>(p) = x;
}

}  // namespace
}  // namespace sgemm
