// layers_linear_instances.hpp -- the kernels' tile widths of one element type.
#pragma once

#include "layers_linear.hpp"

namespace lic {

template <typename F>
int with_linear_tile(int64_t dim, bool vec, F &&f)
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

// A launch of KERNEL over `blocks` blocks of `threads`, in pieces.
template <auto KERNEL, typename ARGS>
int run_linear(ARGS a, int64_t blocks, int threads, int bytes, hipStream_t s)
{
    if (const int rc = allow_lds<KERNEL>(bytes))
        return rc;
    in_pieces(blocks, threads, [&](int64_t first, uint32_t n) {
        a.first = (uint32_t)first;
        a.blocks = n;
        KERNEL<<<xcd_grid(n), threads, bytes, s>>>(a);
    });
    return launched();
}

inline int64_t blocks_of(const LinearArgs &a) { return (int64_t)a.batch * a.heads * a.segments * a.jobs; }
inline int widest(const LinearArgs &a) { return std::max(a.job[0].dim_x, a.job[0].dim_z); }

template <typename T>
int Linear<T>::sweep(LinearArgs a, bool vec, hipStream_t s)
{
    return with_linear_tile(widest(a), vec, [&](auto dt, auto v) {
        using G = Runs<T, dt.value, v.value, 3>;
        bool leaves = false;
        for (int i = 0; i < a.jobs; ++i)
            leaves |= a.job[i].last != nullptr;
        if (leaves)
            return run_linear<linear_sweep<T, dt.value, v.value, kParts<T>>>(a, blocks_of(a), G::kThreads, G::kLds, s);
        return run_linear<linear_sweep<T, dt.value, v.value, kFewParts<T>>>(a, blocks_of(a), G::kThreads, G::kLds, s);
    });
}

template <typename T>
int Linear<T>::states(LinearArgs a, bool vec, hipStream_t s)
{
    return with_linear_tile(widest(a), vec, [&](auto dt, auto v) {
        using G = Runs<T, dt.value, v.value, 2>;
        return run_linear<linear_states<T, dt.value, v.value>>(a, blocks_of(a), G::kThreads, G::kLds, s);
    });
}

template <typename T>
int Linear<T>::decay(DecayArgs a, bool vec, hipStream_t s)
{
    return with_linear_tile(std::max(a.dim, a.value_dim), vec, [&](auto dt, auto v) {
        using G = Runs<T, dt.value, v.value, 4, kDecayWaves<dt.value>>;
        return run_linear<linear_decay<T, dt.value, v.value>>(a, (int64_t)a.batch * a.heads * a.segments, G::kThreads,
                                                              G::kLds, s);
    });
}

}  // namespace lic
