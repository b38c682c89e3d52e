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

template <typename T>
int Linear<T>::sweep(LinearArgs a, bool vec, hipStream_t s)
{
    const int dim = std::max(a.job[0].dim_x, a.job[0].dim_z);
    return with_linear_tile(dim, vec, [&](auto dt, auto v) {
        using G = Sweep<T, dt.value, v.value>;
        constexpr auto kernel = linear_sweep<T, dt.value, v.value>;
        if (const int rc = allow_lds<kernel>(G::kLds))
            return rc;
        const int64_t blocks = (int64_t)a.batch * a.heads * a.jobs;
        in_pieces(blocks, G::kThreads, [&](int64_t first, uint32_t n) {
            a.first = (uint32_t)first;
            a.blocks = n;
            kernel<<<xcd_grid(n), G::kThreads, G::kLds, s>>>(a);
        });
        return launched();
    });
}

template <typename T>
int Linear<T>::decay(DecayArgs a, bool vec, hipStream_t s)
{
    return with_linear_tile(std::max(a.dim, a.value_dim), vec, [&](auto dt, auto v) {
        using G = Decay<T, dt.value, v.value>;
        constexpr auto kernel = linear_decay<T, dt.value, v.value>;
        if (const int rc = allow_lds<kernel>(G::kLds))
            return rc;
        in_pieces((int64_t)a.batch * a.heads, G::kThreads, [&](int64_t first, uint32_t n) {
            a.first = (uint32_t)first;
            a.blocks = n;
            kernel<<<xcd_grid(n), G::kThreads, G::kLds, s>>>(a);
        });
        return launched();
    });
}

}  // namespace lic
