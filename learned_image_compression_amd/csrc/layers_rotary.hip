// layers_rotary.hip -- rotary positions: the tables of cosines and sines, and
// the rotation of queries and keys (its inverse is the gradient).
//
// The rotation is bound by HBM: q and k are read and written once, the tables
// are a small part (a row serves all heads of a token).  A thread turns V pairs
// of one head (two 16-byte loads: V = 8 in 16 bits, V = 4 in 32; V = 4 or 1 where the head
// does not divide) or copies 2 V of the head's other values; neighbouring threads take
// the units of a head, then the heads of a token, so a token's table row is read
// from L1 by all heads but the first.  q and k share one launch.
// Measured, bfloat16: 8 x 32640 positions, 6 heads of 32 of q and k 74 us (5.4 TB/s read and written,
// a large copy 5.0); 16 single tokens, 16 and 4 heads of 64 3.4 us, an empty launch's time.
#include "layers_common.hpp"

namespace lic {
namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
    lic_rotary_args p;
    uint32_t turn_units, units; // units of a head: turning, then copying
    uint32_t all_heads;
    uint64_t total, first; // threads of the call; the launch's first block
};

template <typename T, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a)
{
    using VT = Vec<T, V>;
    const lic_rotary_args &p = a.p;
    const uint64_t id = (a.first + blockIdx.x) * kThreads + threadIdx.x;
    if (id >= a.total)
        return;
    const uint64_t row = id / a.units; // (batch, token, head)
    const uint32_t unit = (uint32_t)(id - row * a.units);
    const uint64_t bs = row / a.all_heads;
    uint32_t head = (uint32_t)(row - bs * a.all_heads);
    const uint64_t b = bs / (uint64_t)p.tokens, s = bs - b * (uint64_t)p.tokens;

    const bool is_q = head < (uint32_t)p.heads;
    if (!is_q)
        head -= (uint32_t)p.heads;
    const int64_t *si = is_q ? p.q_stride : p.k_stride;
    const int64_t *so = is_q ? p.q_out_stride : p.k_out_stride;
    const T *in = static_cast<const T *>(is_q ? p.q : p.k) + b * si[0] + s * si[1] + head * si[2];
    T *out = static_cast<T *>(is_q ? p.q_out : p.k_out) + b * so[0] + s * so[1] + head * so[2];

    const int64_t pos = p.positions ? p.positions[b * p.pos_batch + s] : (int64_t)s;
    const bool there = (uint64_t)pos < (uint64_t)p.table_rows;

    const int half = (int)p.rotary_dim / 2;
    if (unit >= a.turn_units) { // values beyond the rotated part
        const int d0 = (int)p.rotary_dim + (int)(unit - a.turn_units) * 2 * V;
        if (in != out || !there) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (d0 + h * V < p.dim) {
                    VT x = load_at<VT>(in + d0 + h * V);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        x.v[i] = there ? x.v[i] : (T)__builtin_nanf("");
                    store_at(out + d0 + h * V, x);
                }
        }
        return;
    }
    const int j = (int)unit * V;
    const int at0 = INTER ? 2 * j : j, at1 = INTER ? 2 * j + V : half + j;
    const VT x0 = load_at<VT>(in + at0), x1 = load_at<VT>(in + at1);
    float c[V], n[V];
    if (there) {
        constexpr int W = V < 4 ? V : 4;
        const float *ct = p.cos + pos * half + j, *st = p.sin + pos * half + j;
#pragma unroll
        for (int i = 0; i < V; i += W) {
            const auto cv = load_at<Vec<float, W>>(ct + i), sv = load_at<Vec<float, W>>(st + i);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                c[i + w] = cv.v[w];
                n[i + w] = p.inverse ? -sv.v[w] : sv.v[w];
            }
        }
    } else {
        if (p.status)
            *p.status = RANS_E_INDEX;
#pragma unroll
        for (int i = 0; i < V; ++i)
            c[i] = n[i] = __builtin_nanf("");
    }
    VT y0, y1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // pair i: neighbours (interleaved: element 2 i of the 2 V that x0 and x1 hold), or
        // the same place of the two halves
        const int e = 2 * i;
        const float u = up(INTER ? (e < V ? x0.v[e % V] : x1.v[e % V]) : x0.v[i]);
        const float w = up(INTER ? (e + 1 < V ? x0.v[(e + 1) % V] : x1.v[(e + 1) % V]) : x1.v[i]);
        const T t0 = down<T>(u * c[i] - w * n[i]), t1 = down<T>(u * n[i] + w * c[i]);
        if constexpr (INTER) {
            (e < V ? y0 : y1).v[e % V] = t0;
            (e + 1 < V ? y0 : y1).v[(e + 1) % V] = t1;
        } else {
            y0.v[i] = t0;
            y1.v[i] = t1;
        }
    }
    store_at(out + at0, y0);
    store_at(out + at1, y1);
}

struct TableArgs {
    const double *coords;
    float *cos, *sin;
    double base, factor, low, high, original, amplitude;
    uint64_t total, first;
    int axes, pairs;
};

// One thread an angle.  Once for a model, so double precision costs nothing.
__global__ __launch_bounds__(kThreads) void rotary_table_kernel(TableArgs a)
{
    const uint64_t id = (a.first + blockIdx.x) * kThreads + threadIdx.x;
    if (id >= a.total)
        return;
    const uint64_t row = id / (uint32_t)a.pairs;
    const int pair = (int)(id - row * (uint32_t)a.pairs);
    const int n = a.pairs / a.axes, axis = pair / n, j = pair - axis * n;
    double freq = pow(a.base, -(double)j / n);
    if (a.factor != 1.0) {
        double keep = 0.0;
        if (a.high > a.low) {
            const double turns = a.original * freq / 6.283185307179586;
            keep = fmin(1.0, fmax(0.0, (turns - a.low) / (a.high - a.low)));
        }
        freq *= keep + (1.0 - keep) / a.factor;
    }
    double s, c;
    sincos(a.coords[row * (uint32_t)a.axes + axis] * freq, &s, &c);
    a.cos[id] = (float)(c * a.amplitude);
    a.sin[id] = (float)(s * a.amplitude);
}

template <typename T, int V>
int run_rotary(RotaryArgs a, hipStream_t s)
{
    const lic_rotary_args &p = a.p;
    a.turn_units = (uint32_t)(p.rotary_dim / 2 / V);
    a.units = a.turn_units + (uint32_t)((p.dim - p.rotary_dim + 2 * V - 1) / (2 * V));
    a.all_heads = (uint32_t)(p.heads + p.kv_heads);
    const uint64_t rows = (uint64_t)p.batch * p.tokens * a.all_heads; // at most 2^57
    if (rows > (1ull << 48) / a.units)
        return RANS_E_ARG;
    a.total = rows * a.units;
    in_pieces((int64_t)((a.total + kThreads - 1) / kThreads), kThreads, [&](int64_t first, uint32_t blocks) {
        a.first = (uint64_t)first;
        if (p.interleaved)
            rotary_kernel<T, V, true><<<blocks, kThreads, 0, s>>>(a);
        else
            rotary_kernel<T, V, false><<<blocks, kThreads, 0, s>>>(a);
    });
    return launched();
}

// Whether heads divide into V values at once.  Strides and addresses have no part in it: kernels
// of other widths round otherwise (products are combined with sums in one and not in the next).
bool fits(const lic_rotary_args &p, int V) { return (p.rotary_dim / 2) % V == 0 && p.dim % V == 0; }

bool extent(int64_t v, int64_t least, int64_t most) { return v >= least && v <= most; }

}  // namespace
}  // namespace lic

using namespace lic;

extern "C" int lic_rotary_table(const double *coords, int64_t rows, int32_t axes,
                                int32_t rotary_dim, double base, double factor, double low,
                                double high, double original, double amplitude, float *cos,
                                float *sin, hipStream_t hstream)
{
    const auto finite = [](double v) { return v - v == 0.0; };
    if (!extent(rows, 0, 1ll << 31) || axes < 1 || axes > 8 || rotary_dim < 2 ||
        rotary_dim > 65536 || rotary_dim % 2 || (rotary_dim / 2) % axes || !(base > 0.0) ||
        !finite(base) || !(factor > 0.0) || !finite(factor) || !finite(low) || !finite(high) ||
        !(original >= 0.0) || !finite(original) || !finite(amplitude))
        return RANS_E_ARG;
    if (rows == 0)
        return RANS_OK;
    if (!coords || !cos || !sin)
        return RANS_E_ARG;
    TableArgs a{coords, cos, sin, base, factor, low, high, original, amplitude,
                (uint64_t)rows * (uint64_t)(rotary_dim / 2), 0, axes, rotary_dim / 2};
    in_pieces((int64_t)((a.total + kThreads - 1) / kThreads), kThreads, [&](int64_t first, uint32_t blocks) {
        a.first = (uint64_t)first;
        rotary_table_kernel<<<blocks, kThreads, 0, hstream>>>(a);
    });
    return launched();
}

extern "C" int lic_rotary(const lic_rotary_args *args, hipStream_t hstream)
{
    if (!args)
        return RANS_E_ARG;
    const lic_rotary_args &p = *args;
    if (!valid_dtype(p.dtype) || !extent(p.batch, 0, 1ll << 31) || !extent(p.tokens, 0, 1ll << 31) ||
        !extent(p.heads, 1, 65536) || !extent(p.kv_heads, 0, 65536) || !extent(p.dim, 2, 65536) ||
        !extent(p.rotary_dim, 2, p.dim) || p.rotary_dim % 2 || !extent(p.table_rows, 0, 1ll << 40) ||
        p.pos_batch < 0)
        return RANS_E_ARG;
    for (int i = 0; i < 3; ++i)
        if (p.q_stride[i] < 0 || p.k_stride[i] < 0 || p.q_out_stride[i] < 0 ||
            p.k_out_stride[i] < 0)
            return RANS_E_ARG;
    if (p.batch == 0 || p.tokens == 0)
        return RANS_OK;
    if (!p.q || !p.q_out || (p.kv_heads && (!p.k || !p.k_out)) || !p.cos || !p.sin ||
        (!p.positions && p.table_rows < p.tokens) ||
        p.batch > (1ll << 40) / p.tokens)
        return RANS_E_ARG;
    RotaryArgs a{};
    a.p = p;
    return with_dtype(p.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int V = 16 / sizeof(T);
        if (fits(p, V))
            return run_rotary<T, V>(a, hstream);
        if (fits(p, 4)) // 16-bit heads of 24, 40, 72: 8 bytes at once
            return run_rotary<T, 4>(a, hstream);
        return run_rotary<T, 1>(a, hstream);
    });
}

extern "C" const char *lic_layers_target(void) { return "gfx950"; }
