// layers_norm.hip -- group norm with an activation, channels last, forward and
// backward.
//
//   xh = (x - mean_g) rstd_g,  u = w_c xh + b_c,  y = f(u)
//   du = dy f'(u),  S1_c = sum du,  S2_c = sum du xh   (over positions)
//   A_g = sum_c w_c S1_c / m,  B_g = sum_c w_c S2_c / m
//   dx = rstd_g (w_c du - A_g - xh B_g),  db = sum_n S1,  dw = sum_n S2
//      = gain_c du - rstd A - d rstd^2 B  with d = x - mean, gain = w rstd: as it is computed
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
// A thread owns VEC neighbouring channels (16 bytes where they divide the channels) and walks rows, so channel constants stay in registers and neighbouring
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
constexpr int kResident = 512; // threads of a resident block
constexpr int kUnroll = 4;    // vectors in flight of a thread: 64 bytes of loads
constexpr int kJoinAhead = 8; // chunks that a join asks for at once
constexpr int kBlocks = 1024; // of a chunked launch: four a CU

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
    bool past;                          // forward outputs pass the caches
    uint32_t blocks;                    // resident: samples * groups of the launch
    uint32_t first;                     // the launch's first block of the call's
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

// relu, and a sum of squares that rounding may have taken below 0; NaN stays NaN
__device__ __forceinline__ float not_below_zero(float x) { return x < 0.0f ? 0.0f : x; }

__device__ __forceinline__ float fast_exp(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// Phi(u) and the density's e = exp(-u^2 / 2).  The tail Phi(-|u|) is e times a polynomial of degree
// five in t = 1 / (1 + 0.3275911 |u| / sqrt 2) (Abramowitz and Stegun 7.1.26, off by at
// most 1.5e-7), so value and slope share one exponential.
__device__ __forceinline__ void normal_cdf(float u, float &phi, float &e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(u), 0.3275911f * 0.70710678118654752f, 1.0f));
    e = __builtin_amdgcn_exp2f(u * u * (-0.5f * 1.4426950408889634f));
    // half the polynomial
    const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, -0.5f * 1.453152027f),
                                                0.5f * 1.421413741f),
                                        -0.5f * 0.284496736f),
                                0.5f * 0.254829592f);
    phi = 0.5f + copysignf(fmaf(-poly, e, 0.5f), u);
}

template <int ACT>
__device__ __forceinline__ float act_value(float u)
{
    if constexpr (ACT == LIC_ACT_RELU)
        return not_below_zero(u);
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
        return s * fmaf(u, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == LIC_ACT_GELU) {
        float phi, e;
        normal_cdf(u, phi, e);
        return fmaf(u * 0.3989422804014327f, e, phi);
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

// f(vector of each array, row) for a thread's rows: U rows of all arrays are asked for before the
// first is worked on, also at the end of a chunk, where a row a time would cost a memory
// latency each.
template <int U, int ARRAYS, typename V, typename F>
__device__ __forceinline__ void walk(const Place &at, const V *const (&array)[ARRAYS], const int64_t (&row)[ARRAYS],
                                     F &&f)
{
    const int64_t step = at.rows_at_once;
    for (int64_t p = at.row + at.lane_row; p < at.row_end; p += U * step) {
        V v[U][ARRAYS];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * step < at.row_end) {
#pragma unroll
                for (int k = 0; k < ARRAYS; ++k)
                    v[u][k] = load_at<V>(reinterpret_cast<const uint8_t *>(array[k]) + (p + u * step) * row[k]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * step < at.row_end)
                f(v[u], p + u * step);
    }
}

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
//
// Measured, 192 channels of 544 x 960, bfloat16, silu: sums 37 us (5.4 TB/s read), join 5, outputs
// 76 (5.3 TB/s read and written; through the caches sums take 56).  16 x 192 x 64 x 64, backward: sums 18 us (2.8 TB/s), join 4.5,
// outputs 19 (4.0 TB/s); at 50 MB a launch's start and end are a third of it.  8 x 320 x 128 x 128,
// float16, gelu: sums 27, outputs 40, backward 48 and 49 us; without the activation the backward call
// takes 74 us instead of 95, so there arithmetic is a part of what bounds it.
// Eight vectors in flight, or twice or four times the blocks, were no faster.

// Forward: a channel's mean and squares about it over one chunk.
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void norm_partial_forward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const int64_t block = (int64_t)a.first + blockIdx.x;
    const Place at(a, block, VEC);
    const T *base = static_cast<const T *>(a.x) + at.n * a.x_sample;
    float2 s[VEC];
    float shift[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        s[i] = make_float2(0.0f, 0.0f);
    if (at.active) {
        const T *x = base + at.c0;
        const V first = load_at<V>(x + at.row * a.x_row);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            shift[i] = up(first.v[i]);
        const V *const arrays[] = {reinterpret_cast<const V *>(x)};
        const int64_t rows[] = {a.x_row * (int64_t)sizeof(T)};
        walk<kUnroll>(at, arrays, rows, [&](const V(&v)[1], int64_t) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = up(v[0].v[i]) - shift[i];
                s[i].x += d;
                s[i].y += d * d;
            }
        });
    }
    const float count = (float)(at.row_end - at.row);
    const int c_tile = (int)(block % a.tiles) * a.tile_vecs * VEC;
    float2 *part = a.part + ((int64_t)at.n * a.chunks + at.chunk) * a.channels;
    sum_over_rows<VEC>(at, a.tile_vecs, s, [&](int c, float2 t) {
        c += c_tile;
        if (c >= a.channels)
            return;
        const float about = up(base[at.row * a.x_row + c]);
        const float off = t.x / count;
        part[c] = make_float2(about + off, not_below_zero(t.y - t.x * off));
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
    for (int64_t e0 = threadIdx.x; e0 < entries; e0 += kJoinAhead * kThreads) {
        float2 p[kJoinAhead];
        float count[kJoinAhead];
#pragma unroll
        for (int u = 0; u < kJoinAhead; ++u) {
            const int64_t e = least(e0 + u * kThreads, entries - 1), chunk = e / a.per_group;
            p[u] = part[chunk * a.channels + (e - chunk * a.per_group)];
            count[u] = e0 + u * kThreads < entries ? (float)least(a.rows, a.positions - chunk * a.rows) : 0.0f;
            p[u].y = e0 + u * kThreads < entries ? p[u].y : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kJoinAhead; ++u) {
            const float d = p[u].x - about;
            s.x += count[u] * d;
            s.y += p[u].y + count[u] * d * d;
        }
    }
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) {
        const float m = (float)((double)a.positions * a.per_group);
        const float off = s.x / m;
        const float var = not_below_zero(s.y - s.x * off) / m;
        a.mean[(int64_t)n * a.groups + g] = about + off;
        a.rstd[(int64_t)n * a.groups + g] = 1.0f / sqrtf(var + a.eps);
    }
}

// The outputs, last chunk first.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_output_forward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const Place at(a, (int64_t)a.samples * a.chunks * a.tiles - 1 - a.first - blockIdx.x, VEC);
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
    const V *const arrays[] = {reinterpret_cast<const V *>(x)};
    const int64_t rows[] = {a.x_row * (int64_t)sizeof(T)};
    walk<kUnroll>(at, arrays, rows, [&](const V(&v)[1], int64_t p) {
        V o;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            o.v[i] = down<T>(act_value<ACT>((up(v[0].v[i]) - mean[i]) * gain[i] + bias[i]));
        store_at(y + p * a.out_row, o, a.past);
    });
}

// Constants of a thread's channels in the backward kernels: u = gain d + bias with d = x - mean.
template <int VEC>
struct Channels {
    float mean[VEC], gain[VEC], bias[VEC];

    __device__ Channels(const NormArgs &a, int n, int c0)
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int64_t g = (int64_t)n * a.groups + (c0 + i) / a.per_group;
            mean[i] = a.mean[g];
            gain[i] = a.rstd[g] * param(a.weight, a.param_dtype, c0 + i, 1.0f);
            bias[i] = param(a.bias, a.param_dtype, c0 + i, 0.0f);
        }
    }
};

// Backward: a channel's sums of du and du d over one chunk.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_partial_backward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const int64_t block = (int64_t)a.first + blockIdx.x;
    const Place at(a, block, VEC);
    float2 s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        s[i] = make_float2(0.0f, 0.0f);
    if (at.active) {
        const Channels<VEC> ch(a, at.n, at.c0);
        const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample + at.c0;
        const T *dy = static_cast<const T *>(a.dy) + at.n * a.dy_sample + at.c0;
        const V *const arrays[] = {reinterpret_cast<const V *>(x), reinterpret_cast<const V *>(dy)};
        const int64_t rows[] = {a.x_row * (int64_t)sizeof(T), a.dy_row * (int64_t)sizeof(T)};
        walk<kUnroll / 2>(at, arrays, rows, [&](const V(&v)[2], int64_t) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = up(v[0].v[i]) - ch.mean[i];
                const float du = up(v[1].v[i]) * act_slope<ACT>(fmaf(d, ch.gain[i], ch.bias[i]));
                s[i].x += du;
                s[i].y = fmaf(du, d, s[i].y);
            }
        });
    }
    const int c_tile = (int)(block % a.tiles) * a.tile_vecs * VEC;
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
    const float rstd = a.rstd[(int64_t)n * a.groups + g];
    float2 slope = make_float2(0.0f, 0.0f);
    for (int first = 0; first < a.per_group; first += width) {
        const int c = g * a.per_group + first + lane;
        const bool mine = first + lane < a.per_group;
        float2 s = make_float2(0.0f, 0.0f);
        if (mine && way < ways)
            for (int64_t k0 = way; k0 < a.chunks; k0 += kJoinAhead * ways) {
                float2 p[kJoinAhead];
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u)
                    p[u] = part[least(k0 + u * ways, a.chunks - 1) * a.channels + c];
#pragma unroll
                for (int u = 0; u < kJoinAhead; ++u)
                    if (k0 + u * ways < a.chunks) {
                        s.x += p[u].x;
                        s.y += p[u].y;
                    }
            }
        __syncthreads();
        red[t] = s;
        __syncthreads();
        if (way == 0 && mine) {
            for (int w = 1; w < ways; ++w) {
                s.x += red[w * width + lane].x;
                s.y += red[w * width + lane].y;
            }
            s.y *= rstd; // xh = d rstd
            a.totals[(int64_t)n * a.channels + c] = s;
            const float w = param(a.weight, a.param_dtype, c, 1.0f);
            slope.x += w * s.x;
            slope.y += w * s.y;
        }
    }
    slope = block_sum<kThreads>(slope);
    if (t == 0) {
        // as the outputs take them: rstd A and rstd^2 B
        const float m = (float)((double)a.positions * a.per_group);
        a.slopes[(int64_t)n * a.groups + g] = make_float2(rstd * slope.x / m, rstd * rstd * slope.y / m);
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

// dx; the launch's last blocks sum dweight and dbias beside it.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kThreads) void norm_output_backward(NormArgs a)
{
    using V = Vec<T, VEC>;
    const int64_t main_blocks = (int64_t)a.samples * a.chunks * a.tiles, block = (int64_t)a.first + blockIdx.x;
    if (block >= main_blocks) { // the last blocks of the call
        sum_over_samples(a, (int)(block - main_blocks));
        return;
    }
    const Place at(a, main_blocks - 1 - block, VEC);
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
    const V *const arrays[] = {reinterpret_cast<const V *>(x), reinterpret_cast<const V *>(dy)};
    const int64_t rows[] = {a.x_row * (int64_t)sizeof(T), a.dy_row * (int64_t)sizeof(T)};
    walk<kUnroll / 2>(at, arrays, rows, [&](const V(&v)[2], int64_t p) {
        V o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float d = up(v[0].v[i]) - ch.mean[i];
            const float du = up(v[1].v[i]) * act_slope<ACT>(fmaf(d, ch.gain[i], ch.bias[i]));
            o.v[i] = down<T>(fmaf(ch.gain[i], du, fmaf(-d, slope[i].y, -slope[i].x)));
        }
        store_at(dx + p * a.out_row, o);
    });
}

// ---- one launch ------------------------------------------------------------
//
// A block keeps one group of one sample in LDS, each thread its own vectors (of channels of
// the one group) of every rows_at_once-th row.  The blocks of a sample's groups run on one XCD: they
// share its cache lines where a group's channels do not fill one.  A block's latencies bound it (load,
// two sums over the block, store): 1 x 192 x 17 x 30, 32 groups, float 5.3 us, where an empty launch takes 3.7.

struct Resident {
    int n, g, lane_row, rows_at_once, c0, slots;
    bool active;

    __device__ Resident(const NormArgs &a, int vec)
    {
        const uint32_t each = (a.blocks + 7) / 8, place = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
        const uint32_t block = a.first + place;
        active = place < a.blocks;
        n = (int)(block / (uint32_t)a.groups);
        g = (int)(block - (uint32_t)n * a.groups);
        const int t = (int)threadIdx.x, width = a.per_group / vec;
        lane_row = t / width;
        rows_at_once = kResident / width;
        c0 = g * a.per_group + (t - lane_row * width) * vec;
        slots = lane_row < rows_at_once && lane_row < a.positions
                    ? (int)((a.positions - lane_row + rows_at_once - 1) / rows_at_once)
                    : 0;
    }
};

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kResident) void norm_resident_forward(NormArgs a)
{
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) uint8_t lds[];
    V *held = reinterpret_cast<V *>(lds) + threadIdx.x;
    const Resident at(a, VEC);
    if (!at.active)
        return;
    const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample;
    const float shift = up(x[at.g * a.per_group]); // a value of the group
    x += at.c0 + at.lane_row * a.x_row;
    const int64_t step = at.rows_at_once * a.x_row;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < at.slots; ++i) {
        const V v = load_at<V>(x + i * step);
        held[i * kResident] = v;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s.x += up(v.v[e]) - shift;
    }
    const float m = (float)((double)a.positions * a.per_group);
    const float mean = shift + block_sum<kResident>(s).x / m;
    for (int i = 0; i < at.slots; ++i) {
        const V v = held[i * kResident];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float d = up(v.v[e]) - mean;
            s.y += d * d;
        }
    }
    const float rstd = 1.0f / sqrtf(block_sum<kResident>(s).y / m + a.eps);
    if (threadIdx.x == 0) {
        a.mean[(int64_t)at.n * a.groups + at.g] = mean;
        a.rstd[(int64_t)at.n * a.groups + at.g] = rstd;
    }
    if (at.slots == 0)
        return;
    float gain[VEC], bias[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        gain[e] = rstd * param(a.weight, a.param_dtype, at.c0 + e, 1.0f);
        bias[e] = param(a.bias, a.param_dtype, at.c0 + e, 0.0f);
    }
    T *y = static_cast<T *>(a.out) + at.n * a.out_sample + at.c0 + at.lane_row * a.out_row;
    const int64_t out_step = at.rows_at_once * a.out_row;
#pragma unroll 2
    for (int i = 0; i < at.slots; ++i) {
        const V v = held[i * kResident];
        V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            o.v[e] = down<T>(act_value<ACT>((up(v.v[e]) - mean) * gain[e] + bias[e]));
        store_at(y + i * out_step, o);
    }
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(kResident) void norm_resident_backward(NormArgs a)
{
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float2 red[kResident * VEC];
    const Resident at(a, VEC);
    if (!at.active)
        return;
    const int t = (int)threadIdx.x, depth = (int)((a.positions + at.rows_at_once - 1) / at.rows_at_once);
    V *hx = reinterpret_cast<V *>(lds) + t, *hd = hx + depth * kResident;
    const T *x = static_cast<const T *>(a.x) + at.n * a.x_sample + at.c0 + at.lane_row * a.x_row;
    const T *dy = static_cast<const T *>(a.dy) + at.n * a.dy_sample + at.c0 + at.lane_row * a.dy_row;
    const int64_t x_step = at.rows_at_once * a.x_row, dy_step = at.rows_at_once * a.dy_row;
    const int64_t group = (int64_t)at.n * a.groups + at.g;
    const float mean = a.mean[group], rstd = a.rstd[group];
    float gain[VEC], bias[VEC];
    float2 s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const bool mine = at.slots > 0;
        gain[e] = mine ? rstd * param(a.weight, a.param_dtype, at.c0 + e, 1.0f) : 0.0f;
        bias[e] = mine ? param(a.bias, a.param_dtype, at.c0 + e, 0.0f) : 0.0f;
        s[e] = make_float2(0.0f, 0.0f);
    }
#pragma unroll 2
    for (int i = 0; i < at.slots; ++i) {
        const V v = load_at<V>(x + i * x_step);
        const V d = load_at<V>(dy + i * dy_step);
        hx[i * kResident] = v;
        hd[i * kResident] = d;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float off = up(v.v[e]) - mean;
            const float du = up(d.v[e]) * act_slope<ACT>(fmaf(off, gain[e], bias[e]));
            s[e].x += du;
            s[e].y = fmaf(du, off, s[e].y);
        }
    }
    // a group's sums, then each channel's
    float2 slope = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        s[e].y *= rstd; // xh = (x - mean) rstd
        slope.x += gain[e] * s[e].x;
        slope.y += gain[e] * s[e].y;
        red[t * VEC + e] = s[e];
    }
    slope = block_sum<kResident>(slope);
    const float m = (float)((double)a.positions * a.per_group);
    slope.x /= m;
    slope.y *= rstd / m; // the weights in slope hold one rstd already
    for (int c = t; c < a.per_group; c += kResident) {
        float2 sum = red[c];
        for (int r = 1; r < at.rows_at_once; ++r) {
            sum.x += red[r * a.per_group + c].x;
            sum.y += red[r * a.per_group + c].y;
        }
        const int channel = at.g * a.per_group + c;
        if (a.samples > 1) {
            a.totals[(int64_t)at.n * a.channels + channel] = sum;
        } else {
            if (a.dbias)
                put_param(a.dbias, a.param_dtype, channel, sum.x);
            if (a.dweight)
                put_param(a.dweight, a.param_dtype, channel, sum.y);
        }
    }
    T *dx = static_cast<T *>(a.out) + at.n * a.out_sample + at.c0 + at.lane_row * a.out_row;
    const int64_t out_step = at.rows_at_once * a.out_row;
#pragma unroll 2
    for (int i = 0; i < at.slots; ++i) {
        const V v = hx[i * kResident], d = hd[i * kResident];
        V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float off = up(v.v[e]) - mean;
            const float du = up(d.v[e]) * act_slope<ACT>(fmaf(off, gain[e], bias[e]));
            o.v[e] = down<T>(fmaf(gain[e], du, fmaf(-off, slope.y, -slope.x)));
        }
        store_at(dx + i * out_step, o);
    }
}

__global__ __launch_bounds__(kThreads) void norm_samples(NormArgs a) { sum_over_samples(a, (int)blockIdx.x); }

// ---- host ----------------------------------------------------------------

// Channels of a tile: the split of a row into tiles that leaves the fewest of a
// block's threads idle (a row of 160 vectors: 5 tiles of 32 take all 256, one tile 160).
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

// Chunks: about kBlocks blocks if the rows allow it, each thread a whole number of unrolled turns.
void choose_chunks(NormArgs &a)
{
    const int64_t at_once = kThreads / a.tile_vecs, turn = at_once * (a.dy ? kUnroll / 2 : kUnroll);
    const int64_t wanted = kBlocks / ((int64_t)a.samples * a.tiles) + 1;
    a.rows = (a.positions + wanted - 1) / wanted;
    a.rows = (a.rows + turn - 1) / turn * turn;
    a.chunks = (int)((a.positions + a.rows - 1) / a.rows);
}

// The most chunks that any tiling of a row gives.
int64_t most_chunks(int32_t samples) { return kBlocks / (int64_t)samples + 1; }

uint64_t part_bytes(int32_t samples, int32_t channels)
{
    return ((uint64_t)samples * most_chunks(samples) * channels * sizeof(float2) + 255) / 256 * 256;
}

uint64_t totals_bytes(int32_t samples, int32_t channels)
{
    return ((uint64_t)samples * channels * sizeof(float2) + 255) / 256 * 256;
}

// The widest vector that divides the channels.  Strides and addresses have no part in it: it decides
// the order of sums, and the same values have to give the same bits wherever they lie.
template <typename T>
int widest(const NormArgs &a)
{
    for (int vec : {(int)(16 / sizeof(T)), 2})
        if (a.channels % vec == 0)
            return vec;
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

// LDS that a resident block of VEC-wide vectors needs for one array, 0 if it cannot.
template <typename T>
int64_t resident_bytes(const NormArgs &a, int vec)
{
    if (a.per_group % vec || a.per_group / vec > kResident)
        return 0;
    const int64_t at_once = kResident / (a.per_group / vec);
    const int64_t bytes = (a.positions + at_once - 1) / at_once * kResident * vec * (int64_t)sizeof(T);
    return bytes;
}

// The widest vector that also divides a group.
template <typename T>
int resident_vec(const NormArgs &a, int vec)
{
    while (vec > 1 && a.per_group % vec)
        vec = vec > 2 ? 2 : 1;
    return vec;
}

template <typename T, typename F>
int with_vec(int vec, F &&f)
{
    switch (vec) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 1: return f(std::integral_constant<int, 1>{});
    default: return f(std::integral_constant<int, 16 / sizeof(T)>{});
    }
}

// Most LDS that a resident block takes for its values (of 160 KiB; the backward kernel's sums
// take up to 32 more).
constexpr int64_t kMostForward = 128 * 1024, kMostBackward = 96 * 1024;

// One launch or three.  A resident block's time goes with its turns of 512 vectors (0.7 us each;
// a CU takes one block after another), three launches take 10 us and 1.5 us a million values.
// Measured (us, one / three launches, bfloat16): 1 x 192 x 510, 32 groups 5.4 / 12.1; 16 x 192 x 1024
// 11.4 / 13.9; 32 x 1024 x 256 12.8 / 26; 16 x 192 x 4096 36 / 26; 29 x 32 x 4212 30 / 16.
template <typename T>
bool resident_pays(const NormArgs &a, int64_t lds, int vec)
{
    const int64_t arrays = a.dy ? 2 : 1, turns = lds / (arrays * kResident * vec * (int64_t)sizeof(T));
    const double one = 3.5 + 0.7 * (double)(turns * ((a.blocks + 255) / 256));
    const double three = 10.0 + 1.5e-6 * (double)a.samples * (double)a.positions * a.channels;
    return one <= three && lds > 0 && lds <= (a.dy ? kMostBackward : kMostForward);
}

template <typename T>
int run_resident_forward(NormArgs a, int vec, int64_t lds, hipStream_t s)
{
    return with_vec<T>(vec, [&](auto v) {
        return with_act(a.act, [&](auto act) {
            constexpr auto kernel = norm_resident_forward<T, v.value, act.value>;
            if (const int rc = allow_lds<kernel>(kMostForward))
                return rc;
            in_pieces((int64_t)a.samples * a.groups, kResident, [&](int64_t first, uint32_t blocks) {
                a.first = (uint32_t)first, a.blocks = blocks;
                kernel<<<(blocks + 7) / 8 * 8, kResident, (uint32_t)lds, s>>>(a);
            });
            return launched();
        });
    });
}

template <typename T>
int run_resident_backward(NormArgs a, int vec, int64_t lds, hipStream_t s)
{
    return with_vec<T>(vec, [&](auto v) {
        return with_act(a.act, [&](auto act) {
            constexpr auto kernel = norm_resident_backward<T, v.value, act.value>;
            if (const int rc = allow_lds<kernel>(kMostBackward))
                return rc;
            in_pieces((int64_t)a.samples * a.groups, kResident, [&](int64_t first, uint32_t blocks) {
                a.first = (uint32_t)first, a.blocks = blocks;
                kernel<<<(blocks + 7) / 8 * 8, kResident, (uint32_t)lds, s>>>(a);
            });
            if (a.samples > 1 && (a.dweight || a.dbias))
                norm_samples<<<(a.channels + 31) / 32, kThreads, 0, s>>>(a);
            return launched();
        });
    });
}

template <typename T, int VEC>
int run_forward(NormArgs a, hipStream_t s)
{
    choose_tiles(a, VEC);
    choose_chunks(a);
    // 200 MB in and out: 117 us with outputs past the caches, 134 through them
    a.past = 2 * (int64_t)sizeof(T) * a.samples * a.positions * a.channels > kCacheBytes;
    const int64_t blocks = (int64_t)a.samples * a.chunks * a.tiles;
    in_pieces(blocks, kThreads, [&](int64_t first, uint32_t piece) {
        a.first = (uint32_t)first;
        norm_partial_forward<T, VEC><<<piece, kThreads, 0, s>>>(a);
    });
    norm_join_forward<<<dim3(a.groups, a.samples), kThreads, 0, s>>>(a);
    return with_act(a.act, [&](auto act) {
        in_pieces(blocks, kThreads, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first;
            norm_output_forward<T, VEC, act.value><<<piece, kThreads, 0, s>>>(a);
        });
        return launched();
    });
}

template <typename T, int VEC>
int run_backward(NormArgs a, hipStream_t s)
{
    choose_tiles(a, VEC);
    choose_chunks(a);
    const int64_t blocks = (int64_t)a.samples * a.chunks * a.tiles;
    const int more = a.dweight || a.dbias ? (a.channels + 31) / 32 : 0;
    return with_act(a.act, [&](auto act) {
        in_pieces(blocks, kThreads, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first;
            norm_partial_backward<T, VEC, act.value><<<piece, kThreads, 0, s>>>(a);
        });
        norm_join_backward<<<dim3(a.groups, a.samples), kThreads, 0, s>>>(a);
        in_pieces(blocks + more, kThreads, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first;
            norm_output_backward<T, VEC, act.value><<<piece, kThreads, 0, s>>>(a);
        });
        return launched();
    });
}

bool valid_sizes(int32_t samples, int64_t positions, int32_t channels, int32_t groups)
{
    return samples >= 0 && samples <= LIC_MAX_SAMPLES && positions >= 0 &&
           positions <= (1ll << 40) && channels >= 1 && channels <= LIC_MAX_CHANNELS &&
           groups >= 1 && channels % groups == 0 && (int64_t)samples * groups <= 0x7fffffff;
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
    a.blocks = (uint32_t)samples * (uint32_t)groups;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int vec = widest<T>(a), narrow = resident_vec<T>(a, vec);
        const int64_t lds = resident_bytes<T>(a, narrow);
        if (resident_pays<T>(a, lds, narrow))
            return run_resident_forward<T>(a, narrow, lds, hstream);
        return with_vec<T>(vec, [&](auto v) { return run_forward<T, v.value>(a, hstream); });
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
    a.blocks = (uint32_t)samples * (uint32_t)groups;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int vec = widest<T>(a), narrow = resident_vec<T>(a, vec);
        const int64_t lds = 2 * resident_bytes<T>(a, narrow);
        if (resident_pays<T>(a, lds, narrow))
            return run_resident_backward<T>(a, narrow, lds, hstream);
        return with_vec<T>(vec, [&](auto v) { return run_backward<T, v.value>(a, hstream); });
    });
}
