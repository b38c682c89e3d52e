// layers_common.hpp -- element types and small helpers of the network
// operators' kernels (norms, rotary positions, attention, linear attention, clipping).
#pragma once

#include <atomic>
#include <cstdint>
#include <hip/hip_runtime.h>
#include <type_traits>

#include "lic_layers.h"

namespace lic {

using bf16 = __bf16;
using f16 = _Float16;

// smaller and larger of two whole numbers (the mixed overloads of min and max may go
// through double)
__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t most(int64_t a, int64_t b) { return a > b ? a : b; }

// N elements of T as one load or store of at most 16 bytes
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// Global memory is read and written in vectors wherever an element may lie: the hardware takes
// such accesses at any address, and the arithmetic, its order with it, does not depend on one.
template <typename V>
__device__ __forceinline__ V load_at(const void *p)
{
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}

// past: a store that the caches need not keep.  For outputs that would push the inputs out of the 256
// MB last-level cache between two readings of them (kCacheBytes), or out of it for the next reader.
constexpr int64_t kCacheBytes = 256ll << 20;
template <typename V>
__device__ __forceinline__ void store_at(void *p, const V &v, bool past = false)
{
    if constexpr (sizeof(V) == 16) {
        using W = uint32_t __attribute__((ext_vector_type(4), aligned(2)));
        if (past) {
            W w;
            __builtin_memcpy(&w, &v, 16);
            __builtin_nontemporal_store(w, reinterpret_cast<W *>(p));
            return;
        }
    }
    __builtin_memcpy(p, &v, sizeof(V));
}

// rounding to 16 bits is to nearest, ties to even, in both types
template <typename T>
__device__ __forceinline__ float up(T x)
{
    return (float)x;
}

template <typename T>
__device__ __forceinline__ T down(float x)
{
    return (T)x;
}

// The same of a product that rounds by itself first.  float16 has an instruction for product and
// conversion that rounds once, and the compiler takes it in one kernel and not in the next: kernels that
// differ in their loads alone would differ in their results.
template <typename T>
__device__ __forceinline__ T down_apart(float x)
{
    if constexpr (std::is_same<T, f16>::value)
        asm("" : "+v"(x));
    return (T)x;
}

inline bool valid_dtype(int64_t d) { return d == LIC_F32 || d == LIC_F16 || d == LIC_BF16; }
inline int dtype_bytes(int64_t d) { return d == LIC_F32 ? 4 : 2; }

inline bool aligned_to(const void *p, uint64_t n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline int launched() { return hipGetLastError() == hipSuccess ? RANS_OK : RANS_E_HIP; }

// launch(first block, blocks) for all `blocks` of a call.  A launch's threads are counted in 32 bits: more
// than those go out in several launches (each of a multiple of eight blocks but the last).
template <typename F>
void in_pieces(int64_t blocks, int threads, F &&launch)
{
    const int64_t most = 0xffffffffll / threads / 8 * 8;
    for (int64_t first = 0; first < blocks; first += most)
        launch(first, (uint32_t)(blocks - first < most ? blocks - first : most));
}

// Lets KERNEL take `bytes` of LDS, which is more than any may without it, on the current device; each
// device is told once.
template <auto KERNEL>
int allow_lds(int bytes)
{
    static std::atomic<uint64_t> told{0}; // a bit for each of the first 64 devices
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess)
        return RANS_E_HIP;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (told.load(std::memory_order_relaxed) & bit)
        return RANS_OK;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                            bytes) != hipSuccess) {
        (void)hipGetLastError();
        return RANS_E_HIP;
    }
    told.fetch_or(bit, std::memory_order_relaxed);
    return RANS_OK;
}

// f(T{}) for the element type that `dtype` names
template <typename F>
int with_dtype(int64_t dtype, F &&f)
{
    switch (dtype) {
    case LIC_F32: return f(float{});
    case LIC_F16: return f(f16{});
    case LIC_BF16: return f(bf16{});
    default: return RANS_E_ARG;
    }
}

}  // namespace lic
