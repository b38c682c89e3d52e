// layers_norm.hip -- group norm with an activation, channels last, forward and
// backward.
//
//   xh = (x - mean_g) rstd_g,  u = w_c xh + b_c,  y = f(u)
//   du = dy f'(u),  S1_c = sum du,  S2_c = sum du xh   (over positions)
//   A_g = sum_c w_c S1_c / m,  B_g = sum_c w_c S2_c / m
//   dx = rstd_g (w_c du - A_g - xh B_g),  db = sum_n S1,  dw = sum_n S2
//
// HBM bounds all of it.  A group's statistics need all of its values before the
// first output, so x (backward: x and dy) is read twice unless a sample's group
// fits into one CU's LDS:
//
// * one launch (norm_resident_*): a block keeps its groups' values of one sample
//   in LDS between the sums and the outputs.
// * three launches otherwise: per-channel sums of a chunk of rows
//   (norm_partial_*), their join per group (norm_join_*), the outputs
//   (norm_output_*).  The outputs walk the chunks from the last to the first,
//   since the last ones read are what the caches still hold.
//
// A thread owns VEC neighbouring channels (16 bytes where sizes and alignment
// allow) and walks rows, so channel constants stay in registers and neighbouring
// lanes read neighbouring memory; it does not matter where group borders fall.
//
// Sums of squares: about the chunk's first row, a value of the data itself.  If
// that value lies K deviations off, the squares lose about K^2 of their
// precision, but then the variance that they join holds K^2 itself.  Chunks are
// joined by their means and squares about the mean (the parallel variance
// formula), all in 32 bits.
#include <type_traits>

#include "layers_common.hpp"

namespace lic {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4; // rows in flight of a thread: 64 bytes of loads

struct NormArgs {
    const void *x, *dy;
    void *out; // y or dx
    int64_t x_sample, x_row, dy_sample, dy_row, out_sample, out_row;
    const void *weight, *bias;
    void *dweight, *dbias;
    float *mean, *rstd;
    float2 *part;   // [samples][chunks][channels]
    float2 *totals; // backward: [samples][channels] S1, S2
    float2 *slopes; // backward: [samples][groups] A, B
    int64_t positions, rows; // rows of a chunk
    float eps;
    int samples, channels, groups, per_group, param_dtype, act;
    int vecs, tile_vecs, tiles, chunks; // 16-byte vectors of a row, of a tile; tiles of a row
    int bundle;                         // resident: groups of a block
};

__device__ __forceinline__ float param(const void *p, int dtype, int c, float none)
{
    if (!p)
        return none;
    switch (dtype) {
    case LIC_F32: return static_cast<const float *>(p)[c];
    case LIC_F16: return (float)static_cast<const f16 *>(p)[c];
    default: return (float)static_cast<const bf16 *>(p)[c];
    }
}

__device__ __forceinline__ void put_param(void *p, int dtype, int c, float v)
{
    switch (dtype) {
    case LIC_F32: static_cast<float *>(p)[c] = v; break;
    case LIC_F16: static_cast<f16 *>(p)[c] = (f16)v; break;
    default: static_cast<bf16 *>(p)[c] = (bf16)v; break;
    }
}

__device__ __forceinline__ float fast_exp(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// Phi(u) and the density's e = exp(-u^2 / 2).  The tail Phi(-|u|) is e times a polynomial of degree
// five in t = 1 / (1 + 0.3275911 |u| / sqrt 2) (Abramowitz and Stegun 7.1.26, off by at
// most 1.5e-7), so value and slope share one exponential.
__device__ __forceinline__ void normal_cdf(float u, float &phi, float &e)
{
    const float z = fabsf(u) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * z);
    e = fast_exp(-z * z);
    const float poly =
        t * (0.254829592f +
             t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    const float tail = 0.5f * poly * e;
    phi = u < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float u)
{
    if constexpr (ACT == LIC_ACT_RELU)
        return u > 0.0f ? u : u * 0.0f; // NaN stays NaN
    if constexpr (ACT == LIC_ACT_SILU)
        return u * __builtin_amdgcn_rcpf(1.0f + fast_exp(-u));
    if constexpr (ACT == LIC_ACT_GELU) {
        float phi, e;
        normal_cdf(u, phi, e);
        return u * phi;
    }
    return u;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float u)
{
    if constexpr (ACT == LIC_ACT_RELU)
        return u > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == LIC_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp(-u));
        return s + u * s * (1.0f - s);
    }
    if constexpr (ACT == LIC_ACT_GELU) {
        float phi, e;
        normal_cdf(u, phi, e);
        return phi + u * e * 0.3989422804014327f;
    }
    return 1.0f;
}

// What a thread of the chunked kernels works on: sample, chunk, channels, rows.
struct Place {
    int n, chunk, lane_row, rows_at_once, c0;
    int64_t row, row_end;
    bool active;

    __device__ Place(const NormArgs &a, int64_t block, int vec)
    {
        const int tile = (int)(block % a.tiles);
        const int64_t rest = block / a.tiles;
        chunk = (int)(rest % a.chunks);
        n = (int)(rest / a.chunks);
        const int t = (int)threadIdx.x;
        lane_row = t / a.tile_vecs;
        rows_at_once = kThreads / a.tile_vecs;
        const int v = tile * a.tile_vecs + t % a.tile_vecs;
        c0 = v * vec;
        active = lane_row < rows_at_once && v < a.vecs;
        row = (int64_t)chunk * a.rows;
        row_end = min(a.positions, row + a.rows);
    }
};

// Adds up `mine` over the threads that share channels and leaves each
// channel's sum with f(channel in the tile's first .., sum).
template <int VEC, typename F>
__device__ void sum_over_rows(const Place &at, int tile_vecs, const float2 (&mine)[VEC], F &&f)
{
    __shared__ float2 red[kThreads * VEC];
    const int t = (int)threadIdx.x;
    if (at.lane_row < at.rows_at_once) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            red[t * VEC + i] = at.active ? mine[i] : make_float2(0.0f, 0.0f);
    }
    __syncthreads();
    const int width = tile_vecs * VEC;
    for (int c = t; c < width; c += kThreads) {
        float2 s = red[c];
        for (int r = 1; r < at.rows_at_once; ++r) {
            const float2 o = red[r * width + c];
            s.x += o.x;
            s.y += o.y;
        }
        f(c, s);
    }
}

// sum of v over the block's threads, the same for all of them
template <int THREADS>
__device__ float2 block_sum(float2 v)
{
    __shared__ float2 waves[THREADS / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        v.x += __shfl_xor(v.x, d);
        v.y += __shfl_xor(v.y, d);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        waves[threadIdx.x >> 6] = v;
    __syncthreads();
    float2 s = waves[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) {
        s.x += waves[w].x;
        s.y += waves[w].y;
    }
    return s;
}

// ---- three launches ------------------------------------------------------

// Forward: a channel's mean and squares about it over one chunk.
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void norm_partial_forward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const Place at(a, blockIdx.x, VEC);
    const T *base = static_cast<const T *>(a.x) + at.n * a.x_sample;
    float2 s[VEC];
    float shift[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        s[i] = make_float2(0.0f, 0.0f);
    if (at.active) {
        const T *x = base + at.c0;
        const V first = *reinterpret_cast<const V *>(x + at.row * a.x_row);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            shift[i] = up(first.v[i]);
        const int64_t step = at.rows_at_once;
        int64_t p = at.row + at.lane_row;
        for (; p + (kUnroll - 1) * step < at.row_end; p += kUnroll * step) {
            V v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                v[u] = *reinterpret_cast<const V *>(x + (p + u * step) * a.x_row);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = up(v[u].v[i]) - shift[i];
                    s[i].x += d;
                    s[i].y += d * d;
                }
        }
        for (; p < at.row_end; p += step) {
            const V v = *reinterpret_cast<const V *>(x + p * a.x_row);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = up(v.v[i]) - shift[i];
                s[i].x += d;
                s[i].y += d * d;
            }
        }
    }
    const float count = (float)(at.row_end - at.row);
    const int c_tile = (int)(blockIdx.x % a.tiles) * a.tile_vecs * VEC;
    float2 *part = a.part + ((int64_t)at.n * a.chunks + at.chunk) * a.channels;
    sum_over_rows<VEC>(at, a.tile_vecs, s, [&](int c, float2 t) {
        c += c_tile;
        if (c >= a.channels)
            return;
        const float about = up(base[at.row * a.x_row + c]);
        const float off = t.x / count;
        part[c] = make_float2(about + off, fmaxf(t.y - t.x * off, 0.0f));
    });
}

// One block a sample and group: chunks and channels joined to mean and rstd.
__global__ __launch_bounds__(kThreads) void norm_join_forward(NormArgs a)
{
    const int g = blockIdx.x, n = blockIdx.y;
    const float2 *part = a.part + (int64_t)n * a.chunks * a.channels + (int64_t)g * a.per_group;
    const float about = part[0].x;
    const int64_t entries = (int64_t)a.chunks * a.per_group;
    float2 s = make_float2(0.0f, 0.0f);
    for (int64_t e = threadIdx.x; e < entries; e += kThreads) {
        const int64_t chunk = e / a.per_group;
        const float2 p = part[chunk * a.channels + (e - chunk * a.per_group)];
        const float count = (float)min(a.rows, a.positions - chunk * a.rows);
        const float d = p.x - about;
        s.x += count * d;
        s.y += p.y + count * d * d;
    }
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) {
        const float m = (float)((double)a.positions * a.per_group);
        const float off = s.x / m;
        const float var = fmaxf(s.y - s.x * off, 0.0f) / m;
        a.mean[(int64_t)n * a.groups + g] = about + off;
        a.rstd[(int64_t)n * a.groups + g] = 1.0f / sqrtf(var + a.eps);
    }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_output_forward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const Place at(a, (int64_t)gridDim.x - 1 - blockIdx.x, VEC);
    if (!at.active)
        return;
    float mean[VEC], gain[VEC], bias[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int c = at.c0 + i;
        const int64_t g = (int64_t)at.n * a.groups + c / a.per_group;
        mean[i] = a.mean[g];
        gain[i] = a.rstd[g] * param(a.weight, a.param_dtype, c, 1.0f);
        bias[i] = param(a.bias, a.param_dtype, c, 0.0f);
    }
    const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample + at.c0;
    T *y = static_cast<T *>(a.out) + at.n * a.out_sample + at.c0;
    const int64_t step = at.rows_at_once;
    const auto put = [&](const V &v, int64_t p) {
        V o;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            o.v[i] = down<T>(act_value<ACT>((up(v.v[i]) - mean[i]) * gain[i] + bias[i]));
        *reinterpret_cast<V *>(y + p * a.out_row) = o;
    };
    int64_t p = at.row + at.lane_row;
    for (; p + (kUnroll - 1) * step < at.row_end; p += kUnroll * step) {
        V v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = *reinterpret_cast<const V *>(x + (p + u * step) * a.x_row);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            put(v[u], p + u * step);
    }
    for (; p < at.row_end; p += step)
        put(*reinterpret_cast<const V *>(x + p * a.x_row), p);
}

// Constants of a thread's channels in the backward kernels.
template <int VEC>
struct Channels {
    float mean[VEC], rstd[VEC], weight[VEC], bias[VEC];

    __device__ Channels(const NormArgs &a, int n, int c0)
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int64_t g = (int64_t)n * a.groups + (c0 + i) / a.per_group;
            mean[i] = a.mean[g];
            rstd[i] = a.rstd[g];
            weight[i] = param(a.weight, a.param_dtype, c0 + i, 1.0f);
            bias[i] = param(a.bias, a.param_dtype, c0 + i, 0.0f);
        }
    }
};

// Backward: a channel's sums of du and du xh over one chunk.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_partial_backward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const Place at(a, blockIdx.x, VEC);
    float2 s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        s[i] = make_float2(0.0f, 0.0f);
    if (at.active) {
        const Channels<VEC> ch(a, at.n, at.c0);
        const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample + at.c0;
        const T *dy = static_cast<const T *>(a.dy) + at.n * a.dy_sample + at.c0;
        const int64_t step = at.rows_at_once;
        const auto add = [&](const V &v, const V &d) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float xh = (up(v.v[i]) - ch.mean[i]) * ch.rstd[i];
                const float du = up(d.v[i]) * act_slope<ACT>(ch.weight[i] * xh + ch.bias[i]);
                s[i].x += du;
                s[i].y += du * xh;
            }
        };
        constexpr int U = kUnroll / 2; // two arrays are read
        int64_t p = at.row + at.lane_row;
        for (; p + (U - 1) * step < at.row_end; p += U * step) {
            V v[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = *reinterpret_cast<const V *>(x + (p + u * step) * a.x_row);
                d[u] = *reinterpret_cast<const V *>(dy + (p + u * step) * a.dy_row);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                add(v[u], d[u]);
        }
        for (; p < at.row_end; p += step)
            add(*reinterpret_cast<const V *>(x + p * a.x_row),
                *reinterpret_cast<const V *>(dy + p * a.dy_row));
    }
    const int c_tile = (int)(blockIdx.x % a.tiles) * a.tile_vecs * VEC;
    float2 *part = a.part + ((int64_t)at.n * a.chunks + at.chunk) * a.channels;
    sum_over_rows<VEC>(at, a.tile_vecs, s, [&](int c, float2 t) {
        if (c + c_tile < a.channels)
            part[c + c_tile] = t;
    });
}

// One block a sample and group: the chunks' sums joined per channel (totals)
// and, weighted, per group (slopes).
__global__ __launch_bounds__(kThreads) void norm_join_backward(NormArgs a)
{
    __shared__ float2 red[kThreads];
    const int g = blockIdx.x, n = blockIdx.y, t = (int)threadIdx.x;
    const int width = min(a.per_group, kThreads), ways = kThreads / width;
    const int lane = t % width, way = t / width;
    const float2 *part = a.part + (int64_t)n * a.chunks * a.channels;
    float2 slope = make_float2(0.0f, 0.0f);
    for (int first = 0; first < a.per_group; first += width) {
        const int c = g * a.per_group + first + lane;
        const bool mine = first + lane < a.per_group;
        float2 s = make_float2(0.0f, 0.0f);
        if (mine && way < ways)
            for (int64_t k = way; k < a.chunks; k += ways) {
                const float2 p = part[k * a.channels + c];
                s.x += p.x;
                s.y += p.y;
            }
        __syncthreads();
        red[t] = s;
        __syncthreads();
        if (way == 0 && mine) {
            for (int w = 1; w < ways; ++w) {
                s.x += red[w * width + lane].x;
                s.y += red[w * width + lane].y;
            }
            a.totals[(int64_t)n * a.channels + c] = s;
            const float w = param(a.weight, a.param_dtype, c, 1.0f);
            slope.x += w * s.x;
            slope.y += w * s.y;
        }
    }
    slope = block_sum<kThreads>(slope);
    if (t == 0) {
        const float m = (float)((double)a.positions * a.per_group);
        a.slopes[(int64_t)n * a.groups + g] = make_float2(slope.x / m, slope.y / m);
    }
}

// dweight and dbias of 32 channels: totals summed over the samples.
__device__ void sum_over_samples(const NormArgs &a, int block)
{
    __shared__ float2 red[kThreads];
    const int t = (int)threadIdx.x, c = block * 32 + t % 32;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < a.channels)
        for (int n = t / 32; n < a.samples; n += kThreads / 32) {
            const float2 p = a.totals[(int64_t)n * a.channels + c];
            s.x += p.x;
            s.y += p.y;
        }
    red[t] = s;
    __syncthreads();
    if (t < 32 && c < a.channels) {
        for (int w = 1; w < kThreads / 32; ++w) {
            s.x += red[w * 32 + t].x;
            s.y += red[w * 32 + t].y;
        }
        if (a.dbias)
            put_param(a.dbias, a.param_dtype, c, s.x);
        if (a.dweight)
            put_param(a.dweight, a.param_dtype, c, s.y);
    }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_output_backward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const int64_t main_blocks = (int64_t)a.samples * a.chunks * a.tiles;
    if (blockIdx.x >= main_blocks) { // the last blocks of the launch
        sum_over_samples(a, (int)(blockIdx.x - main_blocks));
        return;
    }
    const Place at(a, main_blocks - 1 - blockIdx.x, VEC);
    if (!at.active)
        return;
    const Channels<VEC> ch(a, at.n, at.c0);
    float2 slope[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        slope[i] = a.slopes[(int64_t)at.n * a.groups + (at.c0 + i) / a.per_group];
    const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample + at.c0;
    const T *dy = static_cast<const T *>(a.dy) + at.n * a.dy_sample + at.c0;
    T *dx = static_cast<T *>(a.out) + at.n * a.out_sample + at.c0;
    const int64_t step = at.rows_at_once;
    const auto put = [&](const V &v, const V &d, int64_t p) {
        V o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float xh = (up(v.v[i]) - ch.mean[i]) * ch.rstd[i];
            const float du = up(d.v[i]) * act_slope<ACT>(ch.weight[i] * xh + ch.bias[i]);
            o.v[i] = down<T>(ch.rstd[i] * (ch.weight[i] * du - slope[i].x - xh * slope[i].y));
        }
        *reinterpret_cast<V *>(dx + p * a.out_row) = o;
    };
    constexpr int U = kUnroll / 2;
    int64_t p = at.row + at.lane_row;
    for (; p + (U - 1) * step < at.row_end; p += U * step) {
        V v[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = *reinterpret_cast<const V *>(x + (p + u * step) * a.x_row);
            d[u] = *reinterpret_cast<const V *>(dy + (p + u * step) * a.dy_row);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            put(v[u], d[u], p + u * step);
    }
    for (; p < at.row_end; p += step)
        put(*reinterpret_cast<const V *>(x + p * a.x_row),
            *reinterpret_cast<const V *>(dy + p * a.dy_row), p);
}

// ---- host ----------------------------------------------------------------

// Channels of a tile: the split of a row into tiles that leaves the fewest of a
// block's threads idle (a row of 160 vectors: 3 tiles of 54, 216 threads of 256).
void choose_tiles(NormArgs &a, int vec)
{
    a.vecs = a.channels / vec;
    int best = 0;
    const int least = (a.vecs + kThreads - 1) / kThreads;
    for (int tiles = least; tiles < least + 8; ++tiles) {
        const int tv = (a.vecs + tiles - 1) / tiles;
        const int used = (int)((int64_t)(kThreads / tv) * tv * a.vecs / ((int64_t)tiles * tv));
        if (used > best) {
            best = used;
            a.tile_vecs = tv;
            a.tiles = (a.vecs + tv - 1) / tv;
        }
    }
}

// Chunks: eight blocks a CU if the rows allow it, each row loop at least once unrolled.
void choose_chunks(NormArgs &a)
{
    const int64_t at_once = kThreads / a.tile_vecs;
    const int64_t wanted = 2048 / ((int64_t)a.samples * a.tiles) + 1;
    const int64_t most = (a.positions + at_once * kUnroll - 1) / (at_once * kUnroll);
    const int64_t chunks = wanted < most ? wanted : most;
    a.rows = (a.positions + chunks - 1) / chunks;
    a.chunks = (int)((a.positions + a.rows - 1) / a.rows);
}

// What a workspace has to hold, whatever the vector width: chunks are most with
// the widest tiles' rows, 2048 / samples + 1 of them a tile at most.
int64_t most_chunks(int32_t samples) { return 2048 / (int64_t)samples + 1; }

uint64_t part_bytes(int32_t samples, int32_t channels)
{
    return ((uint64_t)samples * most_chunks(samples) * channels * sizeof(float2) + 255) / 256 * 256;
}

uint64_t totals_bytes(int32_t samples, int32_t channels)
{
    return ((uint64_t)samples * channels * sizeof(float2) + 255) / 256 * 256;
}

// The widest vector that channels, strides and addresses allow.
template <typename T>
int widest(const NormArgs &a)
{
    for (int vec : {(int)(16 / sizeof(T)), 2}) {
        const uint64_t bytes = vec * sizeof(T);
        const auto fits = [&](const void *p, int64_t sample, int64_t row) {
            return !p || (aligned_to(p, bytes) && (a.samples == 1 || sample % vec == 0) &&
                          (a.positions == 1 || row % vec == 0));
        };
        if (a.channels % vec == 0 && fits(a.x, a.x_sample, a.x_row) &&
            fits(a.dy, a.dy_sample, a.dy_row) && fits(a.out, a.out_sample, a.out_row))
            return vec;
    }
    return 1;
}

template <typename F>
int with_act(int act, F &&f)
{
    switch (act) {
    case LIC_ACT_NONE: return f(std::integral_constant<int, LIC_ACT_NONE>{});
    case LIC_ACT_RELU: return f(std::integral_constant<int, LIC_ACT_RELU>{});
    case LIC_ACT_SILU: return f(std::integral_constant<int, LIC_ACT_SILU>{});
    default: return f(std::integral_constant<int, LIC_ACT_GELU>{});
    }
}

template <typename T, int VEC>
int run_forward(NormArgs a, hipStream_t s)
{
    choose_tiles(a, VEC);
    choose_chunks(a);
    const dim3 grid((uint32_t)((int64_t)a.samples * a.chunks * a.tiles));
    norm_partial_forward<T, VEC><<<grid, kThreads, 0, s>>>(a);
    norm_join_forward<<<dim3(a.groups, a.samples), kThreads, 0, s>>>(a);
    return with_act(a.act, [&](auto act) {
        norm_output_forward<T, VEC, act.value><<<grid, kThreads, 0, s>>>(a);
        return launched();
    });
}

template <typename T, int VEC>
int run_backward(NormArgs a, hipStream_t s)
{
    choose_tiles(a, VEC);
    choose_chunks(a);
    const uint32_t blocks = (uint32_t)((int64_t)a.samples * a.chunks * a.tiles);
    const uint32_t more = a.dweight || a.dbias ? (uint32_t)((a.channels + 31) / 32) : 0u;
    return with_act(a.act, [&](auto act) {
        norm_partial_backward<T, VEC, act.value><<<blocks, kThreads, 0, s>>>(a);
        norm_join_backward<<<dim3(a.groups, a.samples), kThreads, 0, s>>>(a);
        norm_output_backward<T, VEC, act.value><<<blocks + more, kThreads, 0, s>>>(a);
        return launched();
    });
}

bool valid_sizes(int32_t samples, int64_t positions, int32_t channels, int32_t groups)
{
    return samples >= 0 && samples <= LIC_MAX_SAMPLES && positions >= 0 &&
           positions <= (1ll << 40) && channels >= 1 && channels <= LIC_MAX_CHANNELS &&
           groups >= 1 && channels % groups == 0;
}

// A row must not overlap the next one; sample strides of inputs may be anything.
bool valid_strides(int64_t sample, int64_t row) { return sample >= 0 && row >= 0; }

}  // namespace
}  // namespace lic

using namespace lic;

extern "C" uint64_t lic_group_norm_workspace_bytes(int32_t samples, int64_t positions,
                                                   int32_t channels, int32_t groups)
{
    if (!valid_sizes(samples, positions, channels, groups) || samples == 0)
        return 0;
    // per-chunk sums, then (backward) the samples' channel totals and group slopes
    return part_bytes(samples, channels) + 2 * totals_bytes(samples, channels);
}

extern "C" int lic_group_norm_forward(const void *x, int64_t x_sample, int64_t x_row,
                                      int32_t samples, int64_t positions, int32_t channels,
                                      int32_t groups, int32_t dtype, const void *weight,
                                      const void *bias, int32_t param_dtype, float eps,
                                      int32_t activation, void *y, int64_t y_sample, int64_t y_row,
                                      float *mean, float *rstd, void *workspace,
                                      uint64_t workspace_bytes, hipStream_t hstream)
{
    if (!valid_sizes(samples, positions, channels, groups) || !valid_dtype(dtype) ||
        !valid_dtype(param_dtype) || activation < 0 || activation > LIC_ACT_GELU ||
        !(eps >= 0.0f) || !valid_strides(x_sample, x_row) || !valid_strides(y_sample, y_row))
        return RANS_E_ARG;
    if (samples == 0 || positions == 0)
        return RANS_OK;
    if (!x || !y || !mean || !rstd)
        return RANS_E_ARG;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < lic_group_norm_workspace_bytes(samples, positions, channels, groups))
        return RANS_E_WORKSPACE;
    NormArgs a{};
    a.x = x, a.x_sample = x_sample, a.x_row = x_row;
    a.out = y, a.out_sample = y_sample, a.out_row = y_row;
    a.weight = weight, a.bias = bias, a.param_dtype = param_dtype;
    a.mean = mean, a.rstd = rstd, a.eps = eps, a.act = activation;
    a.samples = samples, a.positions = positions, a.channels = channels, a.groups = groups;
    a.per_group = channels / groups;
    a.part = static_cast<float2 *>(workspace);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        switch (widest<T>(a)) {
        case 2: return run_forward<T, 2>(a, hstream);
        case 1: return run_forward<T, 1>(a, hstream);
        default: return run_forward<T, 16 / sizeof(T)>(a, hstream);
        }
    });
}

extern "C" int lic_group_norm_backward(const void *dy, int64_t dy_sample, int64_t dy_row,
                                       const void *x, int64_t x_sample, int64_t x_row,
                                       int32_t samples, int64_t positions, int32_t channels,
                                       int32_t groups, int32_t dtype, const void *weight,
                                       const void *bias, int32_t param_dtype, int32_t activation,
                                       const float *mean, const float *rstd, void *dx,
                                       int64_t dx_sample, int64_t dx_row, void *dweight,
                                       void *dbias, void *workspace, uint64_t workspace_bytes,
                                       hipStream_t hstream)
{
    if (!valid_sizes(samples, positions, channels, groups) || samples == 0 || positions == 0 ||
        !valid_dtype(dtype) || !valid_dtype(param_dtype) || activation < 0 ||
        activation > LIC_ACT_GELU || !valid_strides(x_sample, x_row) ||
        !valid_strides(dy_sample, dy_row) || !valid_strides(dx_sample, dx_row) || !dy || !x ||
        !mean || !rstd || !dx)
        return RANS_E_ARG;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < lic_group_norm_workspace_bytes(samples, positions, channels, groups))
        return RANS_E_WORKSPACE;
    NormArgs a{};
    a.x = x, a.x_sample = x_sample, a.x_row = x_row;
    a.dy = dy, a.dy_sample = dy_sample, a.dy_row = dy_row;
    a.out = dx, a.out_sample = dx_sample, a.out_row = dx_row;
    a.weight = weight, a.bias = bias, a.param_dtype = param_dtype;
    a.dweight = dweight, a.dbias = dbias, a.act = activation;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.samples = samples, a.positions = positions, a.channels = channels, a.groups = groups;
    a.per_group = channels / groups;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float2 *>(ws);
    a.totals = reinterpret_cast<float2 *>(ws + part_bytes(samples, channels));
    a.slopes = reinterpret_cast<float2 *>(ws + part_bytes(samples, channels) +
                                          totals_bytes(samples, channels));
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        switch (widest<T>(a)) {
        case 2: return run_backward<T, 2>(a, hstream);
        case 1: return run_backward<T, 1>(a, hstream);
        default: return run_backward<T, 16 / sizeof(T)>(a, hstream);
        }
    });
}
