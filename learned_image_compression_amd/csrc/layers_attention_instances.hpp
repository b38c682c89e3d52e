// layers_attention_instances.hpp -- the kernels' tile widths of one element type.
#pragma once

#include "layers_attention_backward.hpp"
#include "layers_attention_forward.hpp"

namespace lic {

// The head's size rounded up to 32 columns, with 16-byte loads or without them (odd sizes, strides or
// addresses).  Either way the sums of a size are taken in the same order, so the same values give the
// same bits wherever they lie.
template <typename F>
int with_tile(int64_t dim, bool vec, F &&f)
{
    using std::integral_constant;
    const auto width = [&](auto dt) {
        return vec ? f(dt, integral_constant<bool, true>{}) : f(dt, integral_constant<bool, false>{});
    };
    switch ((dim + 31) / 32) {
    case 1: return width(integral_constant<int, 32>{});
    case 2: return width(integral_constant<int, 64>{});
    case 3: return width(integral_constant<int, 96>{});
    default: return width(integral_constant<int, 128>{});
    }
}

// Whether a head's row can be read and written 16 bytes at a time.  (A tile's loads count
// bytes from its first row in 32 bits: 64 rows of less than 2^24 values.)
template <typename T>
bool vector_rows(const lic_attention_args &p, const void *x, const int64_t *stride, int64_t rows, int64_t heads)
{
    constexpr int n = 16 / sizeof(T);
    return !x || (aligned_to(x, 16) && (p.batch == 1 || stride[0] % n == 0) && (rows == 1 || stride[1] % n == 0) &&
                  stride[1] < (1 << 24) &&
                  (heads == 1 || stride[2] % n == 0));
}

template <typename T>
int Attention<T>::forward(AttnArgs a, hipStream_t s)
{
    const lic_attention_args &p = a.p;
    const bool vec = p.dim % (16 / sizeof(T)) == 0 && vector_rows<T>(p, p.q, p.q_stride, p.queries, p.heads) &&
                     vector_rows<T>(p, p.k, p.k_stride, p.keys, p.kv_heads) &&
                     vector_rows<T>(p, p.v, p.v_stride, p.keys, p.kv_heads) &&
                     vector_rows<T>(p, p.out, p.out_stride, p.queries, p.heads);
    return with_tile(p.dim, vec, [&](auto dt, auto v) { return run_forward<T, dt.value, v.value>(a, s); });
}

template <typename T>
int Attention<T>::backward(AttnArgs a, hipStream_t s)
{
    const lic_attention_args &p = a.p;
    const bool vec = p.dim % (16 / sizeof(T)) == 0 && vector_rows<T>(p, p.q, p.q_stride, p.queries, p.heads) &&
                     vector_rows<T>(p, p.k, p.k_stride, p.keys, p.kv_heads) &&
                     vector_rows<T>(p, p.v, p.v_stride, p.keys, p.kv_heads) &&
                     vector_rows<T>(p, p.out, p.out_stride, p.queries, p.heads) &&
                     vector_rows<T>(p, p.dout, p.dout_stride, p.queries, p.heads) &&
                     vector_rows<T>(p, p.dq, p.dq_stride, p.queries, p.heads) &&
                     vector_rows<T>(p, p.dk, p.dk_stride, p.keys, p.kv_heads) &&
                     vector_rows<T>(p, p.dv, p.dv_stride, p.keys, p.kv_heads);
    return with_tile(p.dim, vec, [&](auto dt, auto v) { return run_backward<T, dt.value, v.value>(a, s); });
}

}  // namespace lic
