// layers_common.hpp -- element types and small helpers of the network
// operators' kernels (group norm, rotary positions, attention).
#pragma once

#include <cstdint>
#include <hip/hip_runtime.h>

#include "lic_layers.h"

namespace lic {

using bf16 = __bf16;
using f16 = _Float16;

// N elements of T as one load or store of at most 16 bytes
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

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

inline bool valid_dtype(int64_t d) { return d == LIC_F32 || d == LIC_F16 || d == LIC_BF16; }
inline int dtype_bytes(int64_t d) { return d == LIC_F32 ? 4 : 2; }

inline bool aligned_to(const void *p, uint64_t n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline int launched() { return hipGetLastError() == hipSuccess ? RANS_OK : RANS_E_HIP; }

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
