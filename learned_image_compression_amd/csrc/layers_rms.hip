// layers_rms.hip -- RMS norm with the residual's addition, forward (also with an output
// in 8 bits) and backward.
//
//   h = x + r (rounded),  rstd = 1 / sqrt(mean h^2 + eps),  xh = h rstd,  y = w xh
//   a = w dy,  dx = rstd (a - xh mean(a xh)) + dh,  dw = sum over rows of dy xh
//   8 bits: top = max |y| of the row, out = round(y (most / top))
//
// HBM bounds it: a row is read once and stays in registers, so everything that depends on the
// whole row is in one launch.  A team of lanes takes a row: 2^k lanes of a wave (rows of up to 256
// vectors of 16 bytes, up to four a lane; a wave works on 64 / 2^k rows at once), a block of 256 (up
// to 1024 vectors), and past that a block that reads the row again from the caches (rms_far_*).
// Teams walk rows with the weights (backward: the sums of dw) in registers.  The backward call's sums
// leave each block once and a second launch adds the blocks up, in the blocks' order.
//
// Rows need not divide into vectors: the last vector then ends where the row ends and begins among the
// values of the one before.  Those count once in sums, and are written twice with the same bits; no
// store is before the row's sum, so none is before any lane's loads.
//
// Measured, with the residual: 261120 rows of 192 bfloat16 values forward 68 us (5.9 TB/s of 401 MB), backward
// 78 (5.1 TB/s) and its join 4.6; 65536 rows of 192 float16 values, which the caches hold, 22, 24 and 4; 16320
// rows of 1024 to e4m3 27 us (4.3 TB/s: a row waits for its sum, then for its largest value, before it is stored), to
// int8 27; 16 rows of 1024 4.6 us.  float: 261120 rows of 192 forward 154 us (5.2 TB/s), trained 300 (4.7), 16320 rows
// of 1024 46 and 99.
#include "layers_common.hpp"

namespace lic {
namespace {

constexpr int kRmsThreads = 256;
constexpr int kFarThreads = 1024;
// Blocks of a launch: four a CU, which walk rows and ask for the next one early.  More only begin more often
// (forward, bfloat16, 261120 rows of 192: 85 us with 512, 68 with 1024, 76 with 2048).
constexpr int kBlocks = 1024;

struct RmsArgs {
    lic_rms_norm_args p;
    float *part;          // backward: [blocks][channels] sums of dy xh
    int64_t rows;
    float inverse;        // 1 / channels
    int units, whole;     // vectors of a row; those that begin at a multiple of their size
    int team;             // lanes of a row
    uint32_t blocks;
    bool past;            // y (dx) passes the caches, which the arrays exceed; h does not: the next block reads it
};

__device__ __forceinline__ float weight_at(const lic_rms_norm_args &p, int c)
{
    if (!p.weight)
        return 1.0f;
    switch (p.param_dtype) {
    case LIC_F32: return static_cast<const float *>(p.weight)[c];
    case LIC_F16: return (float)static_cast<const f16 *>(p.weight)[c];
    default: return (float)static_cast<const bf16 *>(p.weight)[c];
    }
}

// The sum (the larger, NaN above all) of a value over a row's team.
template <int THREADS, bool WIDE>
struct Team {
    int lanes;
    float *waves; // of the block, WIDE only

    template <typename F>
    __device__ __forceinline__ float over(float v, F &&f) const
    {
        for (int d = (WIDE ? 64 : lanes) >> 1; d > 0; d >>= 1)
            v = f(v, __shfl_xor(v, d));
        if constexpr (WIDE) {
            __syncthreads();
            if ((threadIdx.x & 63) == 0)
                waves[threadIdx.x >> 6] = v;
            __syncthreads();
            v = waves[0];
#pragma unroll
            for (int w = 1; w < THREADS / 64; ++w)
                v = f(v, waves[w]);
        }
        return v;
    }
    __device__ __forceinline__ float sum(float v) const
    {
        return over(v, [](float a, float b) { return a + b; });
    }
    __device__ __forceinline__ float top(float v) const
    {
        return over(v, [](float a, float b) { return b > a || b != b ? b : a; });
    }
};

// A lane's N vectors of a row: where each begins, and how many of its values are another's.
template <int N, int V, bool TAIL>
struct Vectors {
    int at[N], skip[N];

    __device__ __forceinline__ Vectors(const RmsArgs &a, int lane)
    {
        const int last = (int)a.p.channels - V;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int u = n * a.team + lane;
            at[n] = min(u * V, last);
            skip[n] = u < a.units ? u * V - at[n] : V;
        }
    }
    __device__ __forceinline__ bool there(int n) const { return skip[n] < V; }
    __device__ __forceinline__ bool counts(int n, int i) const { return TAIL ? i >= skip[n] : there(n); }
};

struct At {
    int64_t sample, position;
    __device__ __forceinline__ At(const RmsArgs &a, int64_t row)
        : sample(a.p.samples == 1 ? 0 : row / a.p.positions), position(row - sample * a.p.positions)
    {
    }
    template <typename T>
    __device__ __forceinline__ T *operator()(T *base, const int64_t *stride) const
    {
        return base + sample * stride[0] + position * stride[1];
    }
};

// f(values, place, row, whether it is one) for each of a team's rows, with values = ask(place) that were asked for
// a row ahead; all lanes of a wave go through every turn, since they exchange values.
template <int THREADS, bool WIDE, typename A, typename F>
__device__ __forceinline__ void each_row(const RmsArgs &a, A &&ask, F &&f)
{
    const int t = (int)threadIdx.x, at_once = WIDE ? 1 : THREADS / a.team;
    const int64_t base = (int64_t)blockIdx.x * at_once, step = (int64_t)a.blocks * at_once;
    const int mine = WIDE ? 0 : t / a.team, wave = WIDE ? 0 : (t & ~63) / a.team;
    const auto row = [&](int64_t r) { return least(r + mine, a.rows - 1); };
    if (base + wave >= a.rows)
        return;
    At place(a, row(base));
    auto values = ask(place);
    for (int64_t r = base; r + wave < a.rows; r += step) {
        const At next(a, row(r + step));
        const bool more = r + step + wave < a.rows;
        auto ahead = values;
        if (more)
            ahead = ask(next);
        f(values, place, row(r), r + mine < a.rows);
        values = ahead;
        place = next;
    }
}

// four numbers as e4m3 or whole numbers of a byte
__device__ __forceinline__ uint32_t four_bytes(const float *y, bool e4m3)
{
    uint32_t w = 0;
    if (e4m3) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) // a last bit more than 448 is 448, and NaN stays
            c[i] = y[i] != y[i] ? y[i] : __builtin_amdgcn_fmed3f(y[i], -448.0f, 448.0f);
        w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], (int)w, false);
        w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], (int)w, true);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = y[i] != y[i] ? 0.0f : __builtin_amdgcn_fmed3f(__builtin_rintf(y[i]), -127.0f, 127.0f);
            w |= ((uint32_t)(int)c & 0xffu) << (8 * i);
        }
    }
    return w;
}

__device__ __forceinline__ float most_of(const lic_rms_norm_args &p)
{
    return p.format == LIC_FORMAT_E4M3 ? 448.0f : 127.0f;
}
__device__ __forceinline__ float root(const RmsArgs &a, float squares)
{
    return 1.0f / sqrtf(fmaf(squares, a.inverse, (float)a.p.eps));
}
__device__ __forceinline__ float larger(float top, float y)
{
    const float size = fabsf(y);
    return size > top || size != size ? size : top;
}

template <typename T, int V, int N, int THREADS, bool WIDE, bool TAIL, bool EIGHT>
__global__ __launch_bounds__(THREADS) void rms_forward(RmsArgs a)
{
    using VT = Vec<T, V>;
    __shared__ float waves[THREADS / 64];
    const lic_rms_norm_args &p = a.p;
    const int lane = (int)threadIdx.x & (a.team - 1);
    const Team<THREADS, WIDE> team{a.team, waves};
    const Vectors<N, V, TAIL> vec(a, lane);

    float w[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i)
            w[n][i] = weight_at(p, vec.at[n] + i);
    struct Values {
        VT h[N], o[N];
    };
    const auto ask = [&](const At &place) {
        Values v{};
        const T *x = place(static_cast<const T *>(p.x), p.x_stride);
#pragma unroll
        for (int n = 0; n < N; ++n)
            v.h[n] = load_at<VT>(x + vec.at[n]);
        if (p.residual) {
            const T *residual = place(static_cast<const T *>(p.residual), p.residual_stride);
#pragma unroll
            for (int n = 0; n < N; ++n)
                v.o[n] = load_at<VT>(residual + vec.at[n]);
        }
        return v;
    };
    each_row<THREADS, WIDE>(a, ask, [&](Values &v, const At &place, int64_t row, bool there) {
        VT(&h)[N] = v.h;
        if (p.residual) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    h[n].v[i] = down<T>(up(h[n].v[i]) + up(v.o[n].v[i]));
        }
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = vec.counts(n, i) ? up(h[n].v[i]) : 0.0f;
                s = fmaf(v, v, s);
            }
        const float rstd = root(a, team.sum(s));
        if (there && p.residual) {
            T *sum = place(static_cast<T *>(p.sum), p.sum_stride);
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (vec.there(n))
                    store_at(sum + vec.at[n], h[n]);
        }
        if (there && lane == 0 && p.rstd)
            p.rstd[row] = rstd;
        if constexpr (EIGHT) {
            const bool e4m3 = p.format == LIC_FORMAT_E4M3;
            const float most = most_of(p);
            float y[N][V], top = 1e-30f;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    y[n][i] = up(h[n].v[i]) * rstd * w[n][i];
                    top = larger(top, y[n][i]);
                }
            top = team.top(top);
            const float gain = most / top;
            if (there && lane == 0)
                p.scales[row] = top / most;
            uint8_t *out = place(static_cast<uint8_t *>(p.y), p.y_stride);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if constexpr (V == 1) {
                    const float q[4] = {y[n][0] * gain, 0.0f, 0.0f, 0.0f};
                    if (there && vec.there(n))
                        out[vec.at[n]] = (uint8_t)four_bytes(q, e4m3);
                } else {
                    Vec<uint32_t, V / 4> b;
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        const float q[4] = {y[n][i] * gain, y[n][i + 1] * gain, y[n][i + 2] * gain, y[n][i + 3] * gain};
                        b.v[i / 4] = four_bytes(q, e4m3);
                    }
                    if (there && vec.there(n))
                        store_at(out + vec.at[n], b);
                }
            }
        } else {
            T *out = place(static_cast<T *>(p.y), p.y_stride);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                VT o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.v[i] = down_apart<T>(up(h[n].v[i]) * rstd * w[n][i]);
                if (there && vec.there(n))
                    store_at(out + vec.at[n], o, a.past);
            }
        }
    });
}

template <typename T, int V, int N, int THREADS, bool WIDE, bool TAIL>
__global__ __launch_bounds__(THREADS) void rms_backward(RmsArgs a)
{
    using VT = Vec<T, V>;
    __shared__ float waves[THREADS / 64];
    const lic_rms_norm_args &p = a.p;
    const int lane = (int)threadIdx.x & (a.team - 1);
    const Team<THREADS, WIDE> team{a.team, waves};
    const Vectors<N, V, TAIL> vec(a, lane);

    float w[N][V], dw[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[n][i] = weight_at(p, vec.at[n] + i);
            dw[n][i] = 0.0f;
        }
    struct Values {
        VT h[N], g[N], s[N];
    };
    const auto ask = [&](const At &place) {
        Values v{};
        const T *h = place(static_cast<const T *>(p.x), p.x_stride);
        const T *dy = place(static_cast<const T *>(p.dy), p.dy_stride);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v.h[n] = load_at<VT>(h + vec.at[n]);
            v.g[n] = load_at<VT>(dy + vec.at[n]);
        }
        if (p.dsum) {
            const T *dsum = place(static_cast<const T *>(p.dsum), p.dsum_stride);
#pragma unroll
            for (int n = 0; n < N; ++n)
                v.s[n] = load_at<VT>(dsum + vec.at[n]);
        }
        return v;
    };
    each_row<THREADS, WIDE>(a, ask, [&](const Values &v, const At &place, int64_t row, bool there) {
        const VT(&hv)[N] = v.h, (&gv)[N] = v.g, (&sv)[N] = v.s;
        const float rstd = p.rstd[row];
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float g = up(gv[n].v[i]), xh = up(hv[n].v[i]) * rstd;
                if (there)
                    dw[n][i] = fmaf(g, xh, dw[n][i]);
                if (vec.counts(n, i))
                    s = fmaf(g * w[n][i], xh, s);
            }
        s = team.sum(s) * a.inverse;
        T *dx = place(static_cast<T *>(p.dx), p.dx_stride);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            VT o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = up(hv[n].v[i]) * rstd;
                const float d = rstd * fmaf(-xh, s, up(gv[n].v[i]) * w[n][i]);
                o.v[i] = down_apart<T>(p.dsum ? d + up(sv[n].v[i]) : d);
            }
            if (there && vec.there(n))
                store_at(dx + vec.at[n], o, a.past);
        }
    });
    if (!a.part)
        return;
    float *part = a.part + (int64_t)blockIdx.x * p.channels;
    if constexpr (WIDE) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (vec.counts(n, i))
                    part[vec.at[n] + i] = dw[n][i];
    } else {
        // a wave's rows, then the block's waves
        __shared__ float sums[THREADS / 64][64 * N * V];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                for (int d = a.team; d < 64; d <<= 1)
                    dw[n][i] += __shfl_xor(dw[n][i], d);
                if ((int)(threadIdx.x & 63) < a.team && vec.counts(n, i))
                    sums[threadIdx.x >> 6][vec.at[n] + i] = dw[n][i];
            }
        __syncthreads();
        for (int c = (int)threadIdx.x; c < p.channels; c += THREADS) {
            float s = sums[0][c];
#pragma unroll
            for (int k = 1; k < THREADS / 64; ++k)
                s += sums[k][c];
            part[c] = s;
        }
    }
}

// ---- rows that no block holds in registers --------------------------------
//
// Each thread goes over its vectors again for what depends on the whole row; the row is in the caches then.

// f(first value, values) for a thread's vectors of V
template <int V, typename F>
__device__ __forceinline__ void far_vectors(const RmsArgs &a, F &&f)
{
    const int c = (int)a.p.channels;
    for (int at = (int)threadIdx.x * V; at < c; at += kFarThreads * V)
        f(at, min(V, c - at));
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> far_load(const T *p, int n)
{
    if (n == V)
        return load_at<Vec<T, V>>(p);
    Vec<T, V> v{};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            v.v[i] = p[i];
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void far_store(T *p, const Vec<T, V> &v, int n)
{
    if (n == V) {
        store_at(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            p[i] = v.v[i];
}

template <typename T>
__global__ __launch_bounds__(kFarThreads) void rms_far_forward(RmsArgs a)
{
    constexpr int V = 16 / sizeof(T);
    using VT = Vec<T, V>;
    __shared__ float waves[kFarThreads / 64];
    const lic_rms_norm_args &p = a.p;
    const Team<kFarThreads, true> team{kFarThreads, waves};
    for (int64_t row = blockIdx.x; row < a.rows; row += a.blocks) {
        const At place(a, row);
        const T *h = place(static_cast<const T *>(p.x), p.x_stride);
        float s = 0.0f;
        if (p.residual) {
            const T *x = h, *residual = place(static_cast<const T *>(p.residual), p.residual_stride);
            T *sum = place(static_cast<T *>(p.sum), p.sum_stride);
            far_vectors<V>(a, [&](int at, int n) {
                VT v = far_load<T, V>(x + at, n);
                const VT o = far_load<T, V>(residual + at, n);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v.v[i] = down<T>(up(v.v[i]) + up(o.v[i]));
                    s = fmaf(up(v.v[i]), up(v.v[i]), s);
                }
                far_store<T, V>(sum + at, v, n);
            });
            h = sum; // each thread reads again what it wrote itself
        } else {
            far_vectors<V>(a, [&](int at, int n) {
                const VT v = far_load<T, V>(h + at, n);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    s = fmaf(up(v.v[i]), up(v.v[i]), s);
            });
        }
        const float rstd = root(a, team.sum(s));
        if (threadIdx.x == 0 && p.rstd)
            p.rstd[row] = rstd;
        if (p.format == LIC_FORMAT_NONE) {
            T *out = place(static_cast<T *>(p.y), p.y_stride);
            far_vectors<V>(a, [&](int at, int n) {
                VT v = far_load<T, V>(h + at, n);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < n)
                        v.v[i] = down_apart<T>(up(v.v[i]) * rstd * weight_at(p, at + i));
                far_store<T, V>(out + at, v, n);
            });
            continue;
        }
        const bool e4m3 = p.format == LIC_FORMAT_E4M3;
        const float most = most_of(p);
        float top = 1e-30f;
        far_vectors<V>(a, [&](int at, int n) {
            const VT v = far_load<T, V>(h + at, n);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n)
                    top = larger(top, up(v.v[i]) * rstd * weight_at(p, at + i));
        });
        top = team.top(top);
        const float gain = most / top;
        if (threadIdx.x == 0)
            p.scales[row] = top / most;
        uint8_t *out = place(static_cast<uint8_t *>(p.y), p.y_stride);
        far_vectors<V>(a, [&](int at, int n) {
            const VT v = far_load<T, V>(h + at, n);
            Vec<uint8_t, V> b;
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = i + e < n ? up(v.v[i + e]) * rstd * weight_at(p, at + i + e) * gain : 0.0f;
                const uint32_t word = four_bytes(q, e4m3);
                __builtin_memcpy(&b.v[i], &word, 4);
            }
            far_store<uint8_t, V>(out + at, b, n);
        });
    }
}

template <typename T>
__global__ __launch_bounds__(kFarThreads) void rms_far_backward(RmsArgs a)
{
    constexpr int V = 16 / sizeof(T);
    using VT = Vec<T, V>;
    __shared__ float waves[kFarThreads / 64];
    const lic_rms_norm_args &p = a.p;
    const Team<kFarThreads, true> team{kFarThreads, waves};
    float *part = a.part ? a.part + (int64_t)blockIdx.x * p.channels : nullptr;
    for (int64_t row = blockIdx.x; row < a.rows; row += a.blocks) {
        const At place(a, row);
        const T *h = place(static_cast<const T *>(p.x), p.x_stride);
        const T *dy = place(static_cast<const T *>(p.dy), p.dy_stride);
        const T *dsum = p.dsum ? place(static_cast<const T *>(p.dsum), p.dsum_stride) : nullptr;
        T *dx = place(static_cast<T *>(p.dx), p.dx_stride);
        const float rstd = p.rstd[row];
        float s = 0.0f;
        far_vectors<V>(a, [&](int at, int n) {
            const VT v = far_load<T, V>(h + at, n), g = far_load<T, V>(dy + at, n);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n)
                    s = fmaf(up(g.v[i]) * weight_at(p, at + i), up(v.v[i]) * rstd, s);
        });
        s = team.sum(s) * a.inverse;
        far_vectors<V>(a, [&](int at, int n) {
            const VT v = far_load<T, V>(h + at, n), g = far_load<T, V>(dy + at, n);
            VT o = dsum ? far_load<T, V>(dsum + at, n) : VT{};
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) {
                    const float xh = up(v.v[i]) * rstd;
                    const float d = rstd * fmaf(-xh, s, up(g.v[i]) * weight_at(p, at + i));
                    o.v[i] = down_apart<T>(dsum ? d + up(o.v[i]) : d);
                    if (part) // the block's own, in the order of its rows
                        part[at + i] = fmaf(up(g.v[i]), xh, row == blockIdx.x ? 0.0f : part[at + i]);
                }
            far_store<T, V>(dx + at, o, n);
        });
    }
}

// dw: 32 channels a block, 32 parts at once.
__global__ __launch_bounds__(1024) void rms_join(RmsArgs a)
{
    __shared__ float sums[32][33];
    const int x = (int)threadIdx.x & 31, y = (int)threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x, channels = a.p.channels;
    float s = 0.0f;
    if (c < channels) {
        uint32_t k = (uint32_t)y;
        for (; k + 7 * 32 < a.blocks; k += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = a.part[(int64_t)(k + 32 * i) * channels + c];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s += v[i];
        }
        for (; k < a.blocks; k += 32)
            s += a.part[(int64_t)k * channels + c];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < channels) {
        for (int i = 1; i < 32; ++i)
            s += sums[i][x];
        switch (a.p.param_dtype) {
        case LIC_F32: static_cast<float *>(a.p.dweight)[c] = s; break;
        case LIC_F16: static_cast<f16 *>(a.p.dweight)[c] = (f16)s; break;
        default: static_cast<bf16 *>(a.p.dweight)[c] = (bf16)s; break;
        }
    }
}

// Blocks of the backward call: four a CU, fewer where their sums would be more than 16 MB.
int64_t sum_blocks(int64_t channels)
{
    const int64_t most = (16ll << 20) / (4 * channels);
    return most < 64 ? 64 : most > kBlocks ? kBlocks : most;
}

bool valid(const lic_rms_norm_args *p, bool backward)
{
    const auto in = [](int64_t v, int64_t least, int64_t most) { return v >= least && v <= most; };
    const auto ok = [](const int64_t *s) { return s[0] >= 0 && s[1] >= 0; };
    if (!p || !valid_dtype(p->dtype) || !valid_dtype(p->param_dtype) || !in(p->samples, 0, 1ll << 31) ||
        !in(p->positions, 0, 1ll << 31) || !in(p->channels, 1, LIC_MAX_CHANNELS) ||
        !in(p->format, LIC_FORMAT_NONE, LIC_FORMAT_INT8) || !(p->eps >= 0.0) || !(p->eps < 1e30) || !ok(p->x_stride))
        return false;
    if (p->samples == 0 || p->positions == 0)
        return true;
    if (p->samples > (1ll << 40) / p->positions)
        return false;
    if (backward)
        return p->format == LIC_FORMAT_NONE && p->x && p->rstd && p->dy && p->dx && ok(p->dy_stride) && ok(p->dx_stride) &&
               (!p->dsum || ok(p->dsum_stride));
    return p->x && p->y && ok(p->y_stride) && (!p->residual == !p->sum) &&
           (!p->residual || (ok(p->residual_stride) && ok(p->sum_stride))) &&
           (p->format == LIC_FORMAT_NONE || p->scales);
}

// Rows that lie evenly in all arrays count as those of one sample.
RmsArgs arguments(const lic_rms_norm_args &p, bool backward)
{
    RmsArgs a{};
    a.p = p;
    a.rows = p.samples * p.positions;
    a.inverse = 1.0f / (float)p.channels;
    const int arrays = 2 + (backward ? 1 + (p.dsum != nullptr) : 2 * (p.residual != nullptr));
    a.past = (double)a.rows * (double)p.channels * dtype_bytes(p.dtype) * arrays > (double)kCacheBytes;
    const auto even = [&](const int64_t *s) { return s[0] == s[1] * p.positions; };
    const bool one = even(p.x_stride) &&
                     (backward ? even(p.dy_stride) && even(p.dx_stride) && (!p.dsum || even(p.dsum_stride))
                               : even(p.y_stride) && (!p.residual || (even(p.residual_stride) && even(p.sum_stride))));
    if (one) {
        a.p.positions = a.rows;
        a.p.samples = 1;
    }
    return a;
}

// f(values of a vector, vectors a lane, whether a block takes a row, whether a vector overlaps): the narrowest
// team up to a wave that holds a row with a vector a lane, then up to four vectors a lane (fewer lanes with more
// vectors each wait longer: 16320 rows of 1024 values to e4m3 39 us with four a lane, 29 with two).  far() where no
// block holds it.
template <typename T, typename F, typename G>
int with_team(RmsArgs &a, F &&f, G &&far)
{
    using std::integral_constant;
    constexpr int V = 16 / sizeof(T);
    const int64_t c = a.p.channels;
    const std::false_type no{};
    const std::true_type yes{};
    if (c < V) { // no whole vector: a lane a value
        a.whole = a.units = (int)c;
        a.team = 8;
        return f(integral_constant<int, 1>{}, integral_constant<int, 1>{}, no, no);
    }
    a.whole = (int)(c / V);
    a.units = (int)((c + V - 1) / V);
    if (a.units > 4 * kRmsThreads)
        return far();
    const integral_constant<int, V> vec{};
    const auto go = [&](auto n, auto wide) {
        return a.units == a.whole ? f(vec, n, wide, no) : f(vec, n, wide, yes);
    };
    if (a.units > 256) {
        a.team = kRmsThreads;
        return a.units <= 512 ? go(integral_constant<int, 2>{}, yes) : go(integral_constant<int, 4>{}, yes);
    }
    a.team = 1;
    while (a.team < a.units && a.team < 64)
        a.team *= 2;
    switch ((a.units + a.team - 1) / a.team) {
    case 1: return go(integral_constant<int, 1>{}, no);
    case 2: return go(integral_constant<int, 2>{}, no);
    case 3: return go(integral_constant<int, 3>{}, no);
    default: return go(integral_constant<int, 4>{}, no);
    }
}

// blocks for the rows, at most `most`
uint32_t blocks_of(const RmsArgs &a, int64_t at_once, int64_t most)
{
    const int64_t blocks = (a.rows + at_once - 1) / at_once;
    return (uint32_t)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace lic

using namespace lic;

extern "C" uint64_t lic_rms_norm_workspace_bytes(int64_t samples, int64_t positions, int64_t channels)
{
    if (samples < 1 || positions < 1 || channels < 1 || channels > LIC_MAX_CHANNELS)
        return 0;
    return (uint64_t)(sum_blocks(channels) * channels) * sizeof(float);
}

extern "C" int lic_rms_norm_forward(const lic_rms_norm_args *args, hipStream_t hstream)
{
    if (!valid(args, false))
        return RANS_E_ARG;
    if (args->samples == 0 || args->positions == 0)
        return RANS_OK;
    RmsArgs a = arguments(*args, false);
    return with_dtype(a.p.dtype, [&](auto t) {
        using T = decltype(t);
        return with_team<T>(
            a,
            [&](auto vec, auto n, auto wide, auto tail) {
                constexpr int V = decltype(vec)::value, N = decltype(n)::value;
                constexpr bool WIDE = decltype(wide)::value, TAIL = decltype(tail)::value;
                a.blocks = blocks_of(a, WIDE ? 1 : kRmsThreads / a.team, kBlocks);
                if (a.p.format == LIC_FORMAT_NONE)
                    rms_forward<T, V, N, kRmsThreads, WIDE, TAIL, false><<<a.blocks, kRmsThreads, 0, hstream>>>(a);
                else
                    rms_forward<T, V, N, kRmsThreads, WIDE, TAIL, true><<<a.blocks, kRmsThreads, 0, hstream>>>(a);
                return launched();
            },
            [&] {
                a.blocks = blocks_of(a, 1, 512);
                rms_far_forward<T><<<a.blocks, kFarThreads, 0, hstream>>>(a);
                return launched();
            });
    });
}

extern "C" int lic_rms_norm_backward(const lic_rms_norm_args *args, void *workspace, uint64_t workspace_bytes,
                                     hipStream_t hstream)
{
    if (!valid(args, true))
        return RANS_E_ARG;
    if (args->samples == 0 || args->positions == 0)
        return RANS_OK;
    RmsArgs a = arguments(*args, true);
    if (a.p.dweight) {
        if (!workspace || !aligned_to(workspace, 256) ||
            workspace_bytes < lic_rms_norm_workspace_bytes(args->samples, args->positions, args->channels))
            return RANS_E_WORKSPACE;
        a.part = static_cast<float *>(workspace);
    }
    const int64_t most = a.part ? sum_blocks(a.p.channels) : kBlocks;
    const int rc = with_dtype(a.p.dtype, [&](auto t) {
        using T = decltype(t);
        return with_team<T>(
            a,
            [&](auto vec, auto n, auto wide, auto tail) {
                constexpr int V = decltype(vec)::value, N = decltype(n)::value;
                constexpr bool WIDE = decltype(wide)::value, TAIL = decltype(tail)::value;
                a.blocks = blocks_of(a, WIDE ? 1 : kRmsThreads / a.team, most);
                rms_backward<T, V, N, kRmsThreads, WIDE, TAIL><<<a.blocks, kRmsThreads, 0, hstream>>>(a);
                return launched();
            },
            [&] {
                a.blocks = blocks_of(a, 1, most < 512 ? most : 512);
                rms_far_backward<T><<<a.blocks, kFarThreads, 0, hstream>>>(a);
                return launched();
            });
    });
    if (rc || !a.part)
        return rc;
    rms_join<<<(uint32_t)((a.p.channels + 31) / 32), 1024, 0, hstream>>>(a);
    return launched();
}
