// layers_linear.hpp -- linear attention with a decay for each head: the kernels.
//
//   M_t = g M_(t-1) + y_t z_t',   out_t = s x_t M_t
//
// Runs of C tokens: with M the state before a run and i, j its tokens (0 .. C - 1),
//   out_i = s (sum over j <= i of g^(i-j) (x_i . y_j) z_j + g^(i+1) x_i M),
//   M    <- g^C M + sum over j of g^(C-1-j) y_j z_j'
// so all work is in matrix products and only the states go from run to run.
//
// One kernel (linear_sweep) makes all four results, with the roles x, y, z and the time's direction:
//   out: (q, k, v) forward, from the state         dq: (dout, v, k) forward, from the state transposed
//   dv: (k, q, dout) backward, from dstate         dk: (v, dout, q) backward, from dstate transposed
// (backward in time M holds s sum of g^(i+1) q_i dout_i' of the tokens after a run: the gradient of the
// state between, so the powers of g are one less where it is read and one more where it is written).
//
// A block takes one head of one batch, a wave 32 columns of z: of the state (32 DT of it in its
// accumulators) and of the outputs.  Outputs are formed transposed, so what a token is multiplied by
// (powers of g) is one number a lane, and scores and states are operands of the next product as they
// stand in their accumulators.  Each wave forms the scores for itself: with C = 64 that is a third of the
// products, none of which bounds the kernel, and saves their way through LDS.
#pragma once

#include "layers_attention.hpp"

namespace lic {

struct LinearJob {
    const void *x, *y, *z;
    void *out;
    float *part;        // out, or (where heads share it) each head's part: [batch][head][token][dim_z]
    const float *first; // the state before the tokens (null: 0), element [x's value][z's value]
    float *last;        // and behind them (may be null)
    int64_t x_stride[3], y_stride[3], z_stride[3], out_stride[3]; // batch, row, head
    int64_t first_stride[4], last_stride[4];                      // batch, head, x's value, z's value
    int32_t x_share, y_share, z_share; // heads that share one of x's (y's, z's)
    int32_t dim_x, dim_z;
    int32_t reverse;   // 0, 1: backward in time
    float read, write; // what of s goes to where the state is read, and to where it is written
};

constexpr int kLinearJobs = 3;

struct LinearArgs {
    LinearJob job[kLinearJobs];
    const float *log_decay;
    const int32_t *lengths;
    int64_t tokens;
    int32_t batch, heads, jobs;
    float scale;
    uint32_t blocks, first;
};

// Splits a 32-bit fragment into two operands of T whose sum is it to 2^-17 (bfloat16) or 2^-22.  (float
// is its own operand.)  What is not finite stays in the first alone.
template <typename T>
__device__ __forceinline__ void split(const float (&v)[8], FragV<T> &hi, FragV<T> &lo)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi[i] = down_apart<T>(v[i]);
        const float rest = v[i] - (float)hi[i];
        lo[i] = (T)(not_finite(rest) ? 0.0f : rest);
    }
}

// Half precision: a power of two that brings the largest of finite sizes up (or down) to 2^13, so that what
// is rounded to it for a product keeps its bits; at most 2^MOST.
template <int MOST>
__device__ __forceinline__ float lift_of(float top)
{
    const int e = (int)(__float_as_uint(top) >> 23);
    return e == 0 ? 1.0f : __uint_as_float((uint32_t)min(max(127 + 13 + 127 - e, 127 - 100), 127 + MOST) << 23);
}
constexpr int kStateLift = 120; // of what is multiplied back at once
// of scores: the output's other part is multiplied too, and below 2^-51 a score times a value is
// below half of float16's smallest number
constexpr int kScoreLift = 64;
// 1 / a power of two
__device__ __forceinline__ float inverse_lift(float l) { return __uint_as_float((254u << 23) - __float_as_uint(l)); }
__device__ __forceinline__ float finite_size(float x) { return not_finite(x) ? 0.0f : fabsf(x); }

template <typename T>
constexpr bool kLifts = std::is_same<T, f16>::value;

// Rows of a head on their way to a tile, as Stage, but the first tile row may be the last in memory, and
// rows that are not there become 0: sums go over all of a tile's rows.
template <typename T, int ROWS, int DT, int THREADS, bool VEC>
struct Run {
    using StageT = Stage<T, ROWS, DT, THREADS, VEC>;
    using TileT = Tile<T, ROWS, DT>;
    StageT stage;

    // rows `rows` >= 1 from `base`, the lowest in memory
    __device__ __forceinline__ void fetch(uint8_t *lds, const T *base, int64_t stride, int rows, int dim, bool reverse, int t)
    {
        if constexpr (VEC) {
            const uint32_t first = __builtin_amdgcn_readfirstlane(
                (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + (t & ~63) * 16);
#pragma unroll
            for (int i = 0; i < StageT::kEach; ++i) {
                int row, block, piece;
                StageT::place(i, t, row, block, piece);
                row = min(row, rows - 1);
                const int d = block * 32 + piece * TileT::kPiece;
                const uint32_t at = (uint32_t)(reverse ? rows - 1 - row : row) * (uint32_t)(stride * sizeof(T)) +
                                    d * sizeof(T);
                if (d < dim)
                    load_lds<16>(first + i * THREADS * 16, base, at);
            }
        } else {
#pragma unroll
            for (int i = 0; i < StageT::kEach; ++i) {
                int row, block, piece;
                StageT::place(i, t, row, block, piece);
                const int d = block * 32 + piece * TileT::kPiece;
                const T *p = base + (int64_t)(reverse ? rows - 1 - row : row) * stride + d;
                Vec<T, TileT::kPiece> v;
#pragma unroll
                for (int e = 0; e < TileT::kPiece; ++e)
                    v.v[e] = row < rows && d + e < dim ? p[e] : (T)0.0f;
                stage.r[i] = *reinterpret_cast<const uint4 *>(&v);
            }
        }
    }
    // what fetch() asked for is in LDS (after this and a barrier)
    __device__ __forceinline__ void store(uint8_t *lds, int rows, int t) const
    {
        stage.store(lds, t);
        if constexpr (VEC) {
            if (rows < ROWS) {
#pragma unroll
                for (int i = 0; i < StageT::kEach; ++i) {
                    int row, block, piece;
                    StageT::place(i, t, row, block, piece);
                    if (row >= rows)
                        *reinterpret_cast<uint4 *>(lds + TileT::at(row, block, piece)) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }
};

// A row fragment whose eight values are a column operand's: values 16 kk + 4 h .. and 16 kk + 8 + 4 h .. of `row`.
template <typename T, int ROWS, int DT>
__device__ __forceinline__ FragV<T> row_as_column(const uint8_t *lds, int row, int kk, int h)
{
    using TileT = Tile<T, ROWS, DT>;
    FragV<T> f;
    const int block = kk >> 1;
    if constexpr (sizeof(T) == 2) {
        const int piece = (kk & 1) * 2;
        union {
            uint2 u[2];
            FragV<T> f;
        } u;
        u.u[0] = *reinterpret_cast<const uint2 *>(lds + TileT::at(row, block, piece) + 8 * h);
        u.u[1] = *reinterpret_cast<const uint2 *>(lds + TileT::at(row, block, piece + 1) + 8 * h);
        f = u.f;
    } else {
        using Q = float __attribute__((ext_vector_type(4)));
        const Q a = *reinterpret_cast<const Q *>(lds + TileT::at(row, block, (kk & 1) * 4 + h));
        const Q b = *reinterpret_cast<const Q *>(lds + TileT::at(row, block, (kk & 1) * 4 + 2 + h));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
    return f;
}

// one value of a tile
template <typename T, int ROWS, int DT>
__device__ __forceinline__ float tile_value(const uint8_t *lds, int row, int d)
{
    using TileT = Tile<T, ROWS, DT>;
    return up(*reinterpret_cast<const T *>(lds + TileT::at(row, d >> 5, (d & 31) / TileT::kPiece) +
                                           (d % TileT::kPiece) * sizeof(T)));
}

// Powers of a head's g, g^0 .. g^N, in LDS as a number and the rest to it: formed in 64 bits, since a state
// takes them again with each run.
struct Powers {
    float2 *at;
    __device__ __forceinline__ float operator[](int n) const { return at[n].x; }
    __device__ __forceinline__ void fill(float log_decay, int n, int t, int threads)
    {
        for (int e = t; e <= n; e += threads) {
            const double p = e == 0 ? 1.0 : exp((double)log_decay * e);
            const float hi = (float)p;
            const float lo = (float)(p - (double)hi);
            at[e] = make_float2(hi, not_finite(lo) ? 0.0f : lo);
        }
    }
    // x g^n
    __device__ __forceinline__ float times(float x, float2 p) const { return fmaf(x, p.x, x * p.y); }
};

__device__ __forceinline__ float *part_row(const LinearArgs &a, const LinearJob &p, int b, int head, int64_t row)
{
    return p.part + (((int64_t)b * a.heads + head) * a.tokens + row) * p.dim_z;
}

template <typename T, int DT, bool VEC>
struct Sweep {
    static constexpr int kTiles = sizeof(T) == 2 ? 2 : 1;
    static constexpr int kRun = 32 * kTiles;             // tokens of a run
    static constexpr int kBlocks = DT / 32;              // of 32 columns
    static constexpr int kThreads = 64 * kBlocks;
    static constexpr int kTileBytes = kRun * DT * sizeof(T);
    static constexpr int kLds = 6 * kTileBytes + (kRun + 2) * 8;
    using RunT = Run<T, kRun, DT, kThreads, VEC>;
    using TileT = Tile<T, kRun, DT>;
};

template <typename T>
__device__ __forceinline__ bool odd_values(const FragV<T> &f)
{
    if constexpr (sizeof(T) == 4) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            odd |= not_finite(f[i]);
        return odd;
    } else {
        // an exponent of ones: its lowest bit more carries into the sign's
        constexpr uint32_t ones = std::is_same<T, f16>::value ? 0x7c007c00u : 0x7f807f80u;
        constexpr uint32_t one = std::is_same<T, f16>::value ? 0x04000400u : 0x00800080u;
        union {
            FragV<T> f;
            uint32_t w[4];
        } u;
        u.f = f;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m |= (u.w[i] & ones) + one;
        return (m & 0x80008000u) != 0;
    }
}

// m += sum over a run's tokens of y (z f)', z's columns as fragments, f(token) a token's factor.  The sums are
// exact but for the split of z f.  The accumulators are settled.
template <typename T, typename TileT, int ND, int N, typename F>
__device__ __forceinline__ void add_outer(float16v (&m)[ND], const uint8_t *yt, const FragV<T> (&zf)[N], int lane, F &&f)
{
    const int h = lane >> 5;
    float zw[N][8], top = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            zw[j][e] = (float)zf[j][e] * f(16 * j + (e & 3) + 4 * h + 8 * (e >> 2));
            if constexpr (kLifts<T>)
                top = fmaxf(top, finite_size(zw[j][e]));
        }
    const auto products = [&](float16v(&to)[ND]) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            FragV<T> hi, lo;
            split<T>(zw[j], hi, lo);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const FragV<T> yf = TileT::col_frag(yt, 16 * j, d, lane);
                to[d] = mma(yf, hi, to[d]);
                if constexpr (sizeof(T) == 2)
                    to[d] = mma(yf, lo, to[d]);
            }
        }
        settle<T>();
    };
    if constexpr (kLifts<T>) { // a column's power of two, multiplied back before the sum with m
        const float lift = lift_of<kStateLift>(pair_max(top)), back = inverse_lift(lift);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                zw[j][e] *= lift;
        float16v sum[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d)
            sum[d] = zero16();
        products(sum);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m[d][i] = fmaf(sum[d][i], back, m[d][i]);
    } else {
        products(m);
    }
}

// z's columns of a run
template <typename T, typename TileT, int N>
__device__ __forceinline__ void columns(FragV<T> (&zf)[N], const uint8_t *zt, int block, int lane)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        zf[j] = TileT::col_frag(zt, 16 * j, block, lane);
}

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(2 * DT) void linear_sweep(LinearArgs a)
{
    using G = Sweep<T, DT, VEC>;
    using RunT = typename G::RunT;
    using TileT = typename G::TileT;
    constexpr int ND = G::kBlocks, TILES = G::kTiles, C = G::kRun;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t at = xcd_order(blockIdx.x, a.blocks);
    if (at >= a.blocks)
        return;
    const uint32_t which = a.first + at;
    const LinearJob &p = a.job[which % (uint32_t)a.jobs];
    const uint32_t line = which / (uint32_t)a.jobs;
    const int b = (int)(line / (uint32_t)a.heads), head = (int)(line - (uint32_t)b * a.heads);
    const int t = (int)threadIdx.x, lane = t & 63, c = lane & 31, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const bool reverse = p.reverse != 0, works = 32 * w < p.dim_z;

    const int tokens = (int)a.tokens;
    const int len = a.lengths ? min(max(a.lengths[b], 0), tokens) : tokens;
    const T *x = head_row<T>(p.x, p.x_stride, b, 0, head / p.x_share);
    const T *y = head_row<T>(p.y, p.y_stride, b, 0, head / p.y_share);
    const T *z = head_row<T>(p.z, p.z_stride, b, 0, head / p.z_share);

    const auto tile = [&](int buffer, int which) { return lds + (3 * buffer + which) * G::kTileBytes; };
    Powers g{reinterpret_cast<float2 *>(lds + 6 * G::kTileBytes)};
    g.fill(a.log_decay[head], C, t, G::kThreads);
    for (int i = 0; i < 6; ++i)
        RunT::StageT::clear(lds + i * G::kTileBytes, i % 3 == 2 ? p.dim_z : p.dim_x, t);

    // the state, columns 32 w + c
    float16v m[ND];
    const int col = 32 * w + c;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        m[d] = zero16();
        if (p.first && col < p.dim_z) {
            const float *first = p.first + b * p.first_stride[0] + head * p.first_stride[1] + col * p.first_stride[3];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 32 * d + acc_row(i, h);
                if (row < p.dim_x)
                    m[d][i] = first[row * p.first_stride[2]];
            }
        }
    }

    RunT rx, ry, rz;
    const auto rows_of_run = [&](int k) { return min(C, len - k * C); };
    // the lowest row of run k
    const auto low = [&](int k) { return reverse ? len - k * C - rows_of_run(k) : k * C; };
    const auto fetch = [&](int k, int buffer) {
        const int n = rows_of_run(k);
        const int64_t row = low(k);
        rx.fetch(tile(buffer, 0), x + row * p.x_stride[1], p.x_stride[1], n, p.dim_x, reverse, t);
        ry.fetch(tile(buffer, 1), y + row * p.y_stride[1], p.y_stride[1], n, p.dim_x, reverse, t);
        rz.fetch(tile(buffer, 2), z + row * p.z_stride[1], p.z_stride[1], n, p.dim_z, reverse, t);
    };
    const int runs = (len + C - 1) / C;
    __syncthreads(); // the powers, and the tiles' unused columns
    if (runs > 0)
        fetch(0, 0);

    // g^(i - j) of a tile on the diagonal and of the one before it
    float16v weight[TILES];
#pragma unroll
    for (int n = 0; n < TILES; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = 32 * n + c - acc_row(i, h);
            weight[n][i] = e >= 0 ? g[max(e, 0)] * a.scale : 0.0f;
        }

    for (int k = 0; k < runs; ++k) {
        const int n = rows_of_run(k), buffer = k & 1;
        uint8_t *xt = tile(buffer, 0), *yt = tile(buffer, 1), *zt = tile(buffer, 2);
        rx.store(xt, n, t);
        ry.store(yt, n, t);
        rz.store(zt, n, t);
        __syncthreads();
        if (k + 1 < runs)
            fetch(k + 1, buffer ^ 1);
        if (!works)
            continue;

        // z's columns, as they are and as the state takes them
        FragV<T> zf[2 * TILES];
        columns<T, TileT>(zf, zt, w, lane);
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 2 * TILES; ++j)
            odd |= odd_values<T>(zf[j]);
        odd = __any(odd);

        // x M, the state rounded to an operand
        FragV<T> mf[2 * ND];
        float m_lift = 1.0f;
        if constexpr (kLifts<T>) {
            float top = 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = fmaxf(top, finite_size(m[d][i]));
#pragma unroll
            for (int s = 32; s > 0; s >>= 1)
                top = fmaxf(top, __shfl_xor(top, s));
            m_lift = lift_of<kStateLift>(top);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            float16v lifted = m[d];
            if constexpr (kLifts<T>) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    lifted[i] *= m_lift;
            }
            mf[2 * d] = operand<T>(lifted, 0);
            mf[2 * d + 1] = operand<T>(lifted, 1);
        }
        float16v o[TILES];
        float o_lift[TILES];
#pragma unroll
        for (int it = 0; it < TILES; ++it) {
            FragV<T> xf[2 * ND];
#pragma unroll
            for (int kk = 0; kk < 2 * ND; ++kk)
                xf[kk] = row_as_column<T, C, DT>(xt, 32 * it + c, kk, h);
            o[it] = zero16();
#pragma unroll
            for (int kk = 0; kk < 2 * ND; ++kk)
                o[it] = mma(mf[kk], xf[kk], o[it]);
            // scores, tokens before along the rows
            float16v s[TILES];
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                s[jt] = zero16();
#pragma unroll
                for (int kk = 0; kk < 2 * ND; ++kk)
                    s[jt] = mma(row_as_column<T, C, DT>(yt, 32 * jt + c, kk, h), xf[kk], s[jt]);
            }
            float top = 0.0f;
#pragma unroll
            for (int jt = 0; jt <= it; ++jt)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // a later token's score counts for nothing, whatever it is
                    const bool seen = jt < it || acc_row(i, h) <= c;
                    s[jt][i] = seen ? s[jt][i] * weight[it - jt][i] : 0.0f;
                    if constexpr (kLifts<T>)
                        top = fmaxf(top, finite_size(s[jt][i]));
                }
            o_lift[it] = 1.0f;
            if constexpr (kLifts<T>) {
                o_lift[it] = lift_of<kScoreLift>(pair_max(top));
#pragma unroll
                for (int jt = 0; jt <= it; ++jt)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[jt][i] *= o_lift[it];
            }
            const int i = 32 * it + c;
            float f = g[i + (reverse ? 0 : 1)] * p.read;
            if constexpr (kLifts<T>)
                f *= o_lift[it] * inverse_lift(m_lift);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[it][r] *= f;
#pragma unroll
            for (int jt = 0; jt < it; ++jt)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    o[it] = mma(zf[2 * jt + half], operand<T>(s[jt], half), o[it]);
            if (!odd) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    o[it] = mma(zf[2 * it + half], operand<T>(s[it], half), o[it]);
                settle<T>();
            } else {
                // a later token's NaN times its score of 0 would be NaN here: what is not finite is left
                // out of the product and added where it is seen
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    FragV<T> fine = zf[2 * it + half];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        fine[e] = not_finite((float)fine[e]) ? (T)0.0f : fine[e];
                    o[it] = mma(fine, operand<T>(s[it], half), o[it]);
                }
                settle<T>();
                for (int j = 0; j < 32; ++j) {
                    // the score of token j and this lane's, from the lane and register that hold it
                    const int from = (j >> 2) & 1, i0 = 4 * (j >> 3) + (j & 3);
                    float score = 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        score = r == i0 ? s[it][r] : score;
                    score = __shfl(score, c + 32 * from);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float v = tile_value<T, C, DT>(zt, 32 * it + j, 32 * w + acc_row(r, h));
                        if (j <= c && not_finite(v))
                            o[it][r] += score * v;
                    }
                }
            }
        }

        // the state behind the run
        const float2 whole = g.at[n];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m[d][i] = g.times(m[d][i], whole);
        add_outer<T, TileT>(m, yt, zf, lane, [&](int j) { return g[max(n - 1 - j, 0) + (reverse ? 1 : 0)] * p.write; });
        const int64_t row0 = low(k);
#pragma unroll
        for (int it = 0; it < TILES; ++it) {
            const int i = 32 * it + c;
            const int64_t row = row0 + (reverse ? n - 1 - i : i);
            const float f = kLifts<T> ? inverse_lift(o_lift[it]) : 1.0f;
            if (i >= n)
                continue;
            if (p.part)
                put_column<float, VEC>(part_row(a, p, b, head, row), o[it], f, w, h, p.dim_z);
            else
                put_column<T, VEC>(head_row<T>(p.out, p.out_stride, b, row, head), o[it], f, w, h, p.dim_z);
        }
    }

    if (!works)
        return;
    // rows behind the last token
    for (int row = len + h; row < tokens; row += 2)
        if (col < p.dim_z) {
            if (p.part)
                part_row(a, p, b, head, row)[col] = 0.0f;
            else
                head_row<T>(p.out, p.out_stride, b, row, head)[col] = (T)0.0f;
        }
    if (p.last && col < p.dim_z) {
        float *last = p.last + b * p.last_stride[0] + head * p.last_stride[1] + col * p.last_stride[3];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 32 * d + acc_row(i, h);
                if (row < p.dim_x)
                    last[row * p.last_stride[2]] = m[d][i];
            }
    }
}

// ---- the decay's gradient ----------------------------------------------------
//
// A pair of tokens s <= t has g to the power t - s in it, so the gradient of log g counts the steps:
//   sum over pairs of (t - s) w_ts,  w_ts = scale g^(t-s) (q_t . k_s) (dout_t . v_s)
// and the same with t + 1 for the state given, n - 1 - s for the gradient of the state left.  Going forward,
// with S the state and T = dS / dlog g before a run:
//   pairs within it: elementwise, from the two score matrices in 32 bits
//   the others: <T, U> + <S, V>,  U = scale sum_i g^(i+1) q_i dout_i',  V the same with i + 1 in front
//   T <- g^C (T + C S) + sum_j (C-1-j) g^(C-1-j) k_j v_j'
// All of these are sums over tokens of an exact operand and one that is split in two, so nothing is rounded
// to 16 bits on its way.  At the end <T, dstate> counts the steps of what is left over.
struct DecayArgs {
    const void *q, *k, *v, *dout;
    const float *state, *dstate;
    float *sums; // [batch][heads]
    int64_t q_stride[3], k_stride[3], v_stride[3], dout_stride[3], state_stride[3], dstate_stride[3];
    const float *log_decay;
    const int32_t *lengths;
    int64_t tokens;
    int32_t batch, heads, share, dim, value_dim;
    float scale;
    uint32_t blocks, first;
};

template <typename T, int DT, bool VEC>
struct Decay {
    using S = Sweep<T, DT, VEC>;
    static constexpr int kRun = 32;
    static constexpr int kBlocks = DT / 32, kThreads = 64 * kBlocks;
    static constexpr int kTileBytes = kRun * DT * sizeof(T);
    static constexpr int kLds = 8 * kTileBytes + (kRun + 2) * 8 + kBlocks * 8;
    using RunT = Run<T, kRun, DT, kThreads, VEC>;
    using TileT = Tile<T, kRun, DT>;
};

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(2 * DT) void linear_decay(DecayArgs a)
{
    using G = Decay<T, DT, VEC>;
    using RunT = typename G::RunT;
    using TileT = typename G::TileT;
    constexpr int ND = G::kBlocks, C = G::kRun;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t at = xcd_order(blockIdx.x, a.blocks);
    if (at >= a.blocks)
        return;
    const uint32_t line = a.first + at;
    const int b = (int)(line / (uint32_t)a.heads), head = (int)(line - (uint32_t)b * a.heads), kv = head / a.share;
    const int t = (int)threadIdx.x, lane = t & 63, c = lane & 31, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tokens = (int)a.tokens;
    const int len = a.lengths ? min(max(a.lengths[b], 0), tokens) : tokens;
    const T *src[4] = {head_row<T>(a.q, a.q_stride, b, 0, head), head_row<T>(a.k, a.k_stride, b, 0, kv),
                       head_row<T>(a.v, a.v_stride, b, 0, kv), head_row<T>(a.dout, a.dout_stride, b, 0, head)};
    const int64_t step[4] = {a.q_stride[1], a.k_stride[1], a.v_stride[1], a.dout_stride[1]};
    const int dims[4] = {a.dim, a.dim, a.value_dim, a.value_dim};

    const auto tile = [&](int buffer, int which) { return lds + (4 * buffer + which) * G::kTileBytes; };
    Powers g{reinterpret_cast<float2 *>(lds + 8 * G::kTileBytes)};
    float *waves = reinterpret_cast<float *>(lds + 8 * G::kTileBytes + (C + 2) * 8);
    g.fill(a.log_decay[head], C, t, G::kThreads);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        RunT::StageT::clear(lds + i * G::kTileBytes, dims[i % 4], t);

    float16v s[ND], u[ND];
    const int col = 32 * w + c;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        s[d] = u[d] = zero16();
        if (a.state && col < a.value_dim) {
            const float *state = a.state + b * a.state_stride[0] + head * a.state_stride[1] + col;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 32 * d + acc_row(i, h);
                if (row < a.dim)
                    s[d][i] = state[row * a.state_stride[2]];
            }
        }
    }

    RunT run[4];
    const auto rows_of_run = [&](int k) { return min(C, len - k * C); };
    const auto fetch = [&](int k, int buffer) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            run[i].fetch(tile(buffer, i), src[i] + (int64_t)k * C * step[i], step[i], rows_of_run(k), dims[i], false, t);
    };
    const int runs = (len + C - 1) / C;
    __syncthreads();
    if (runs > 0)
        fetch(0, 0);
    float sum = 0.0f;
    for (int k = 0; k < runs; ++k) {
        const int n = rows_of_run(k), buffer = k & 1;
        const uint8_t *qt = tile(buffer, 0), *kt = tile(buffer, 1), *vt = tile(buffer, 2), *dt = tile(buffer, 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            run[i].store(tile(buffer, i), n, t);
        __syncthreads();
        if (k + 1 < runs)
            fetch(k + 1, buffer ^ 1);
        if (k % ND == w) { // pairs within the run: the waves take turns
            float16v x = zero16(), y = zero16();
#pragma unroll
            for (int kk = 0; kk < 2 * ND; ++kk) {
                x = mma(TileT::row_frag(kt, c, kk, h), TileT::row_frag(qt, c, kk, h), x);
                y = mma(TileT::row_frag(vt, c, kk, h), TileT::row_frag(dt, c, kk, h), y);
            }
            settle<T>();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = c - acc_row(i, h);
                if (e > 0)
                    sum = fmaf(x[i] * y[i], a.scale * (float)e * g[max(e, 0)], sum);
            }
        }
        if (32 * w >= a.value_dim)
            continue;
        float16v m[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d)
            m[d] = zero16();
        FragV<T> df[2];
        columns<T, TileT>(df, dt, w, lane);
        add_outer<T, TileT>(m, qt, df, lane, [&](int i) { return a.scale * g[i + 1]; });
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sum = fmaf(m[d][i], u[d][i], sum);
#pragma unroll
        for (int d = 0; d < ND; ++d)
            m[d] = zero16();
        add_outer<T, TileT>(m, qt, df, lane, [&](int i) { return a.scale * (float)(i + 1) * g[i + 1]; });
        const float2 whole = g.at[n];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sum = fmaf(m[d][i], s[d][i], sum);
                u[d][i] = g.times(fmaf((float)n, s[d][i], u[d][i]), whole);
                s[d][i] = g.times(s[d][i], whole);
            }
        columns<T, TileT>(df, vt, w, lane);
        add_outer<T, TileT>(u, kt, df, lane, [&](int j) { return (float)max(n - 1 - j, 0) * g[max(n - 1 - j, 0)]; });
        add_outer<T, TileT>(s, kt, df, lane, [&](int j) { return g[max(n - 1 - j, 0)]; });
    }
    if (a.dstate && col < a.value_dim) {
        const float *dstate = a.dstate + b * a.dstate_stride[0] + head * a.dstate_stride[1] + col;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 32 * d + acc_row(i, h);
                if (row < a.dim)
                    sum = fmaf(u[d][i], dstate[row * a.dstate_stride[2]], sum);
            }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        sum += __shfl_xor(sum, d);
    if (lane == 0)
        waves[w] = sum;
    __syncthreads();
    if (t == 0) {
        for (int i = 1; i < ND; ++i)
            sum += waves[i];
        a.sums[line] = sum;
    }
}

// Per element type; defined in one translation unit each (layers_linear_<type>.hip).
template <typename T>
struct Linear {
    static int sweep(LinearArgs a, bool vec, hipStream_t s);
    static int decay(DecayArgs a, bool vec, hipStream_t s);
};

}  // namespace lic
