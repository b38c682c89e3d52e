// layers_linear.hpp -- linear attention with a decay for each head: the kernels.
//
//   M_t = g M_(t-1) + y_t z_t',   out_t = s x_t M_t
//
// Runs of C = 32 tokens: with M the state before a run and i, j its tokens (0 .. C - 1),
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
// A block takes a segment of the tokens of one head of one batch, a wave 32 columns of z: of the state (its
// DT rows in the accumulators) and of the outputs.  Outputs are formed transposed, so what a token is
// multiplied by (a power of g) is one number a lane, and scores and states are operands of the next
// product as they stand in their accumulators (in 16-bit types as parts that add up to them).  Each wave forms the scores for itself, which saves their
// way through LDS.  Where heads are few, tokens are split into segments: linear_states forms what each adds
// to the state, linear_scan goes over the segments, and the sweep begins each with its state.
#pragma once

#include "layers_attention.hpp"

namespace lic {

struct LinearJob {
    const void *x, *y, *z; // (the states' kernel reads y and z)
    void *out;
    float *part;        // out, or (where heads share it) each head's part: [batch][head][token][dim_z]
    const float *first; // the state before the tokens (null: 0), element [x's value][z's value]
    float *last;        // and behind them (may be null)
    float *starts;      // where the tokens are split: the state before each segment, [batch][head][segment],
                        // as a wave's accumulators hold it (StateImage)
    int64_t x_stride[3], y_stride[3], z_stride[3], out_stride[3]; // batch, row, head
    int64_t first_stride[4], last_stride[4];                      // batch, head, x's value, z's value
    int32_t x_share, y_share, z_share; // heads that share one of x's (y's, z's)
    int32_t dim_x, dim_z;
    int32_t reverse;   // 0, 1: backward in time
    int32_t turned;    // 0, 1: `starts` holds the state transposed
    float read, write; // what of s goes to where the state is read, and to where it is written
};

constexpr int kLinearJobs = 3;

struct LinearArgs {
    LinearJob job[kLinearJobs];
    const float *log_decay;
    const int32_t *lengths;
    int64_t tokens;
    int32_t batch, heads, jobs;
    int32_t segments, each;  // of the tokens, and tokens of one
    int32_t start_floats;    // of one segment's state
    float scale;
    uint32_t blocks, first;
};

// A segment of a batch's tokens: [from, to), of which `len` are in use.
struct Segment {
    int from, to, len;
    __device__ __forceinline__ Segment(const int32_t *lengths, int b, int tokens, int each, int index)
    {
        const int all = lengths ? min(max(lengths[b], 0), tokens) : tokens;
        from = index * each;
        to = min(tokens, from + each);
        len = min(max(all - from, 0), each);
    }
};

// Operands of T whose sum is a 32-bit fragment: three of bfloat16 hold its 24 bits (two are off by up to 2^-17 of it,
// eight times what 32-bit sums are allowed here), two of float16 are off by up to 2^-23.  float is its own operand.
template <typename T>
constexpr int kParts = std::is_same<T, float>::value ? 1 : std::is_same<T, f16>::value ? 2 : 3;
// For what only outputs of T see: the scores and the state on their way into the products that form them, and a
// state that does not leave the call.  Two parts of bfloat16 are off by up to 2^-17, a 512th of what the output's own
// rounding may be.  (One alone made errors of 0.0023 of an output where its rounding makes 0.0017: 8160 tokens of 2
// x 16 heads of 64 51 us with one, 58 with two, 63 with three; 8160 trained by 16 heads of 128 370, 410 and 464.)
template <typename T>
constexpr int kFewParts = std::is_same<T, float>::value ? 1 : 2;

// odd: some are not finite; those stay in the first part alone.
template <typename T, int PARTS>
__device__ __forceinline__ void split(const float (&v)[8], FragV<T> (&part)[PARTS], bool odd)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float rest = v[i];
#pragma unroll
        for (int n = 0; n < PARTS; ++n) {
            part[n][i] = n + 1 < PARTS || PARTS == 1 ? down_apart<T>(rest) : (T)rest;
            rest -= (float)part[n][i];
        }
    }
    if (odd) {
#pragma unroll
        for (int n = 1; n < PARTS; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[n][i] = not_finite((float)part[0][i]) ? (T)0.0f : part[n][i];
    }
}

// Half precision: a power of two that brings the largest of finite sizes up (or down) to 2^13, so that what
// is rounded to it for a product keeps its bits; at most 2^120, whose inverse is a normal number.
__device__ __forceinline__ float lift_of(float top)
{
    const int e = (int)(__float_as_uint(top) >> 23);
    return e == 0 ? 1.0f : __uint_as_float((uint32_t)min(127 + 13 + 127 - e, 127 + 120) << 23);
}
// 1 / a power of two
__device__ __forceinline__ float inverse_lift(float l) { return __uint_as_float((254u << 23) - __float_as_uint(l)); }
__device__ __forceinline__ float finite_size(float x) { return not_finite(x) ? 0.0f : fabsf(x); }

template <typename T>
constexpr bool kLifts = std::is_same<T, f16>::value;

// Eight of an accumulator's values (half 0 or 1 of them), in half precision times a power of two, as parts.
template <typename T, int PARTS>
__device__ __forceinline__ void split_half(const float16v &m, int half, float lift, FragV<T> (&part)[PARTS], bool odd)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = kLifts<T> ? m[8 * half + i] * lift : m[8 * half + i];
    split<T, PARTS>(v, part, odd);
}
__device__ __forceinline__ bool any_odd(const float16v &v)
{
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        odd |= not_finite(v[i]);
    return odd;
}

// Rows of a head on their way to a tile, as Stage, run after run; backward in time the last in memory
// becomes the tile's first.  The last run may have fewer rows: it ends where the tile ends, with rows of 0
// before it, since sums go over all of a tile's rows and what a token is multiplied by is then the same in
// every run.
template <typename T, int ROWS, int DT, int THREADS, bool VEC>
struct Run {
    using StageT = Stage<T, ROWS, DT, THREADS, VEC>;
    using TileT = Tile<T, ROWS, DT>;
    StageT stage;
    const T *base, *next; // the segment's first row, and the next run's lowest
    int64_t stride;
    int dim;
    bool reverse;
    uint32_t from[VEC ? StageT::kEach : 1]; // bytes to a thread's pieces from the run's lowest row

    __device__ __forceinline__ Run(const T *base, int64_t stride, int dim, bool reverse, int len, int t)
        : base(base), next(base + (reverse ? max(len - ROWS, 0) : 0) * stride), stride(stride), dim(dim), reverse(reverse)
    {
        aim(ROWS, t);
    }
    // rows before a short run repeat its first
    __device__ __forceinline__ void aim(int rows, int t)
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < StageT::kEach; ++i) {
                int row, block, piece;
                StageT::place(i, t, row, block, piece);
                row = max(row - (ROWS - rows), 0);
                from[i] = (uint32_t)(reverse ? rows - 1 - row : row) * (uint32_t)(stride * sizeof(T)) +
                          (block * 32 + piece * TileT::kPiece) * sizeof(T);
            }
        }
    }

    // the next run, of `rows` >= 1 rows
    __device__ __forceinline__ void fetch(uint8_t *lds, int rows, int t)
    {
        if (rows < ROWS) {
            next = reverse ? base : next;
            aim(rows, t);
        }
        if constexpr (VEC) {
            const uint32_t first = __builtin_amdgcn_readfirstlane(
                (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + (t & ~63) * 16);
            if (dim == DT) {
#pragma unroll
                for (int i = 0; i < StageT::kEach; ++i)
                    load_lds<16>(first + i * THREADS * 16, next, from[i]);
            } else {
#pragma unroll
                for (int i = 0; i < StageT::kEach; ++i) {
                    int row, block, piece;
                    StageT::place(i, t, row, block, piece);
                    if (block * 32 + piece * TileT::kPiece < dim)
                        load_lds<16>(first + i * THREADS * 16, next, from[i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < StageT::kEach; ++i) {
                int row, block, piece;
                StageT::place(i, t, row, block, piece);
                const int d = block * 32 + piece * TileT::kPiece;
                row -= ROWS - rows;
                const T *p = next + (int64_t)(reverse ? rows - 1 - row : row) * stride + d;
                Vec<T, TileT::kPiece> v;
#pragma unroll
                for (int e = 0; e < TileT::kPiece; ++e)
                    v.v[e] = row >= 0 && d + e < dim ? p[e] : (T)0.0f;
                stage.r[i] = *reinterpret_cast<const uint4 *>(&v);
            }
        }
        next += reverse ? -ROWS * stride : ROWS * stride;
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
                    if (row < ROWS - rows)
                        *reinterpret_cast<uint4 *>(lds + TileT::at(row, block, piece)) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }
};

// The state's rows stand in its accumulators so that eight of them are neighbours as an operand, like a row
// fragment's values: row `acc` of an accumulator is row state_row(acc) of its 32.  The products that form
// the state take y's columns in that order (column c of them is state_row(c)).
__host__ __device__ __forceinline__ constexpr int state_row(int acc)
{
    return (acc & 0x13) | (acc & 4) << 1 | (acc & 8) >> 1;
}

// y's columns 32 block + state_row(l % 32), as Tile::col_frag
template <typename T, typename TileT>
__device__ __forceinline__ FragV<T> state_columns(const uint8_t *lds, int row0, int block, int lane)
{
    FragV<T> f;
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
        // the middle two of the four fours of columns that 16 lanes ask for, the other way round
        const int j = lane & 15;
        const int row = row0 + 4 * h + (j >> 2);
        const int piece = ((lane >> 4) & 1) * 2 + (j & 1);
        using Lds = __attribute__((address_space(3))) short4v;
        const auto read = [&](int r) {
            const uint8_t *p = lds + TileT::at(r, block, piece) + ((j & 2) >> 1) * 8;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds *)(__attribute__((address_space(3))) void *)p);
        };
        union {
            short4v s[2];
            FragV<T> f;
        } u;
        u.s[0] = read(row);
        u.s[1] = read(row + 8);
        f = u.f;
    } else {
        const int c = state_row(lane & 31);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = row0 + acc_row(i, h);
            f[i] = *reinterpret_cast<const float *>(lds + TileT::at(row, block, c >> 2) + (c & 3) * 4);
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

// Powers of a head's g, g^0 .. g^N, in LDS.
struct Powers {
    float *at;
    __device__ __forceinline__ float operator[](int n) const { return at[n]; }
    // (the exponent's rounding would be off by as much of a power as the exponent is of 2^24)
    __device__ __forceinline__ void fill(float log_decay, int n, int t, int threads)
    {
        for (int e = t; e <= n; e += threads) {
            const float x = log_decay * (float)e, g = expf(x), rest = fmaf(log_decay, (float)e, -x);
            at[e] = e == 0 ? 1.0f : not_finite(x) ? g : fmaf(g, rest, g);
        }
    }
};

// What a state is multiplied by from run to run, g^32.  Its rounding to 32 bits would grow with the
// number of runs, so every sixteenth run takes it with the sixteen errors' sum: what a sixteenth
// of that is off by stays, 2^-29 a run, and what came in since is off by 2^-21 at most, once.
struct Step {
    float whole, mended;
    __device__ __forceinline__ Step(float log_decay, int n)
    {
        const double p = exp((double)log_decay * n);
        whole = (float)p;
        const float rest = (float)(p - (double)whole);
        mended = not_finite(rest) ? whole : fmaf(16.0f, rest, whole);
    }
    __device__ __forceinline__ float at(int run) const { return (run & 15) == 15 ? mended : whole; }
};

__device__ __forceinline__ float *part_row(const LinearArgs &a, const LinearJob &p, int b, int head, int64_t row)
{
    return p.part + (((int64_t)b * a.heads + head) * a.tokens + row) * p.dim_z;
}

constexpr int kRun = 32; // tokens of a run

// What the kernels hold of their tiles: TILES of kRun rows for each of two runs, and g's powers.  WAVES for each
// 32 columns.
template <typename T, int DT, bool VEC, int TILES, int WAVES = 1>
struct Runs {
    static constexpr int kBlocks = DT / 32; // of 32 columns
    static constexpr int kThreads = 64 * kBlocks * WAVES;
    static constexpr int kTileBytes = kRun * DT * sizeof(T);
    static constexpr int kPowers = 2 * TILES * kTileBytes;
    static constexpr int kFactors = kPowers + (kRun + 4) * 4; // of a token where the state takes it in
    static constexpr int kSteps = kFactors + 4 * kRun * 4; // of four tiles: what a pair so many tokens apart counts
    static constexpr int kBacks = kSteps + (TILES == 4 ? (2 * kRun + 4) * 4 : 0); // of three tiles in half precision:
                                                                                   // a wave's columns'
    static constexpr int kLds = kBacks + (TILES == 3 && kLifts<T> ? 32 * kBlocks * 4 : 0);
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

// Tokens' factors where the state takes them in, as a column operand holds the tokens.
struct Factors {
    float f[2][8];

    __device__ __forceinline__ Factors(const float *of, int h)
    {
        using V4 = float __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const V4 v = *reinterpret_cast<const V4 *>(of + 8 * j + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[j >> 1][4 * (j & 1) + e] = v[e];
        }
    }
};

// z's columns of a run
template <typename T, typename TileT>
__device__ __forceinline__ void columns(FragV<T> (&zf)[2], const uint8_t *zt, int block, int lane)
{
#pragma unroll
    for (int j = 0; j < 2; ++j)
        zf[j] = TileT::col_frag(zt, 16 * j, block, lane);
}

// z f of a run's tokens as operands that are their parts, in half precision times a power of two for each column.
template <typename T, int PARTS>
struct Taken {
    FragV<T> part[2][PARTS];
    float back;

    // odd: some of z f are not finite
    __device__ __forceinline__ Taken(const FragV<T> (&zf)[2], const Factors &f, bool odd) : back(1.0f)
    {
        float zw[2][8], top = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                zw[j][e] = (float)zf[j][e] * f.f[j][e];
                if constexpr (kLifts<T>)
                    top = fmaxf(top, finite_size(zw[j][e]));
            }
        if constexpr (kLifts<T>) {
            const float lift = lift_of(pair_max(top));
            back = inverse_lift(lift);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    zw[j][e] *= lift;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            split<T, PARTS>(zw[j], part[j], odd);
    }
    // m + sum over the tokens of y (z f)' / back, y's columns as fragments
    __device__ __forceinline__ float16v times(const FragV<T> (&yf)[2], float16v m) const
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int n = 0; n < PARTS; ++n)
                m = mma(yf[j], part[j][n], m);
        return m;
    }
};

// m += sum over a run's tokens of y (z f)'.  The sums are exact but for the split of z f; the accumulators are
// settled.
template <typename T, typename TileT, int ND, int PARTS>
__device__ __forceinline__ void add_outer(float16v (&m)[ND], const uint8_t *yt, const Taken<T, PARTS> &z, int lane)
{
    float16v sum[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const FragV<T> yf[2] = {state_columns<T, TileT>(yt, 0, d, lane), state_columns<T, TileT>(yt, 16, d, lane)};
        if constexpr (kLifts<T>)
            sum[d] = z.times(yf, zero16());
        else
            m[d] = z.times(yf, m[d]);
    }
    settle<T>();
    if constexpr (kLifts<T>) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m[d][i] = fmaf(sum[d][i], z.back, m[d][i]);
    }
}

template <int ND>
__device__ __forceinline__ void decay(float16v (&m)[ND], float power)
{
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            m[d][i] *= power;
}

// A wave's columns of a state to or from memory: at(row) is where row `row` of its lane's column is.
template <int ND, typename F>
__device__ __forceinline__ void each_row_of_state(int rows, int h, F &&f)
{
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 32 * d + state_row(acc_row(i, h));
            if (row < rows)
                f(d, i, row);
        }
}

// Where a segment's state lies in scratch memory: as the accumulators of the waves hold it, so a lane reads and
// writes 16 bytes at a time, a wave 1 KiB.  For a DT x DT state, four rows a vector:
//   vector ((d * 4 + i / 4) * ND + w) * 64 + lane
template <int ND>
struct StateImage {
    static constexpr int kFloats = 1024 * ND * ND;
    using V4 = Vec<float, 4>;

    static __device__ __forceinline__ int at(int d, int fours, int w, int lane) { return ((d * 4 + fours) * ND + w) * 64 + lane; }
    template <typename F>
    static __device__ __forceinline__ void each(int w, int lane, F &&f)
    {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f(d, i, at(d, i, w, lane));
    }
    static __device__ __forceinline__ void load(float16v (&m)[ND], const float *image, int w, int lane)
    {
        each(w, lane, [&](int d, int i, int at) {
            const V4 v = load_at<V4>(image + 4 * at);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m[d][4 * i + e] = v.v[e];
        });
    }
    static __device__ __forceinline__ void store(const float16v (&m)[ND], float *image, int w, int lane)
    {
        each(w, lane, [&](int d, int i, int at) {
            V4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v.v[e] = m[d][4 * i + e];
            store_at(image + 4 * at, v);
        });
    }
    // The transposed state: its column 32 w + c is row c of the image's rows' block w, and its rows are
    // columns there.
    static __device__ __forceinline__ void load_turned(float16v (&m)[ND], const float *image, int w, int lane)
    {
        const int c = lane & 31, h = lane >> 5, acc = state_row(c); // its own inverse
        const float *mine = image + 4 * (acc & 4 ? 32 : 0) + (acc & 3);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m[d][i] = mine[4 * at(w, acc >> 3, d, state_row(acc_row(i, h)))];
    }
};

// Which job, batch, head and segment a block has; neighbours share a head's tokens.
struct Work {
    int job, b, head, segment;
    int64_t line;
    __device__ __forceinline__ Work(uint32_t which, int jobs, int segments, int heads)
    {
        const uint32_t rest = which / (uint32_t)jobs;
        job = (int)(which - rest * (uint32_t)jobs);
        line = rest / (uint32_t)segments;
        segment = (int)(rest - (uint32_t)line * (uint32_t)segments);
        b = (int)((uint32_t)line / (uint32_t)heads);
        head = (int)((uint32_t)line - (uint32_t)b * (uint32_t)heads);
    }
};

__device__ __forceinline__ float *start_of(const LinearArgs &a, const LinearJob &p, int64_t line, int segment)
{
    return p.starts + (line * a.segments + segment) * a.start_floats;
}

// ---- outputs -------------------------------------------------------------------
//
// Latency bounds a run: its tiles arrive in LDS while the run before is computed, and where there are blocks enough two
// waves a SIMD (three for heads of 32 in 16 bits: 32 x 256 tokens of 6 heads trained 72 us with two, 68 with three;
// wider heads spill with three, 8160 tokens trained by 16 heads of 128 410 us and 502) fill each other's waits; the split
// into segments leaves few heads of 32 or of 128 one.  Measured, bfloat16: 16 heads of 128 on 4, 8160 tokens: out 66 us, dq, dk
// and dv in one launch 138 (278 MB, 2.0 TB/s); 2 x 16 heads of 64 on 4, 8160 tokens 35 us; 6 heads of 32, 32640 tokens
// 20.
//
// PARTS of what a state takes in: all of them where the state leaves the call, with the precision of 32-bit sums.
template <typename T, int DT, bool VEC, int PARTS>
__global__ __launch_bounds__(2 * DT, sizeof(T) == 2 && DT == 32 ? 3 : 2) void linear_sweep(LinearArgs a)
{
    using G = Runs<T, DT, VEC, 3>;
    using RunT = typename G::RunT;
    using TileT = typename G::TileT;
    constexpr int ND = G::kBlocks, C = kRun, FEW = kFewParts<T>;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t at = xcd_order(blockIdx.x, a.blocks);
    if (at >= a.blocks)
        return;
    const Work work(a.first + at, a.jobs, a.segments, a.heads);
    const LinearJob &p = a.job[work.job];
    const int b = work.b, head = work.head;
    const int t = (int)threadIdx.x, lane = t & 63, c = lane & 31, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6), col = 32 * w + c;
    const int dim_z = p.dim_z;
    const bool reverse = p.reverse != 0, works = 32 * w < dim_z;
    const Segment seg(a.lengths, b, (int)a.tokens, a.each, work.segment);
    const int len = seg.len, runs = (len + C - 1) / C;

    const auto tile = [&](int buffer, int which) { return lds + (3 * buffer + which) * G::kTileBytes; };
    RunT rx(head_row<T>(p.x, p.x_stride, b, seg.from, head / p.x_share), p.x_stride[1], p.dim_x, reverse, len, t);
    RunT ry(head_row<T>(p.y, p.y_stride, b, seg.from, head / p.y_share), p.y_stride[1], p.dim_x, reverse, len, t);
    RunT rz(head_row<T>(p.z, p.z_stride, b, seg.from, head / p.z_share), p.z_stride[1], dim_z, reverse, len, t);
    const auto rows_of_run = [&](int k) { return min(C, len - k * C); };
    const auto fetch = [&](int k, int buffer) {
        const int n = rows_of_run(k);
        rx.fetch(tile(buffer, 0), n, t);
        ry.fetch(tile(buffer, 1), n, t);
        rz.fetch(tile(buffer, 2), n, t);
    };
    if (runs > 0)
        fetch(0, 0);
    for (int i = 0; i < 6; ++i) // what no load writes
        RunT::StageT::clear(lds + i * G::kTileBytes, i % 3 == 2 ? p.dim_z : p.dim_x, t);

    // the state before the segment
    float16v m[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
        m[d] = zero16();
    if (a.segments > 1) {
        const float *start = start_of(a, p, work.line, work.segment);
        if (p.turned)
            StateImage<ND>::load_turned(m, start, w, lane);
        else
            StateImage<ND>::load(m, start, w, lane);
    } else if (col < p.dim_z && p.first) {
        const float *first = p.first + b * p.first_stride[0] + head * p.first_stride[1] + col * p.first_stride[3];
        each_row_of_state<ND>(p.dim_x, h, [&](int d, int i, int row) { m[d][i] = first[row * p.first_stride[2]]; });
    }

    Powers g{reinterpret_cast<float *>(lds + G::kPowers)};
    float *factors = reinterpret_cast<float *>(lds + G::kFactors);
    float *backs = reinterpret_cast<float *>(lds + G::kBacks) + 32 * w; // half precision: 1 / the columns' powers of two
    const float log_decay = a.log_decay[head];
    g.fill(log_decay, C, t, G::kThreads);
    const Step step(log_decay, C);
    __syncthreads();
    if (t < C)
        factors[t] = g[C - 1 - t + (reverse ? 1 : 0)] * p.write;
    // s g^(i - j), tokens j along the rows
    float16v weight;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        weight[i] = g[max(c - acc_row(i, h), 0)] * a.scale;
    const float come = g[c + (reverse ? 0 : 1)] * p.read;

    // A run's outputs go out during the next: the wait for its tiles would wait for them too.  A lane's row of
    // a whole run, and the step to the next run's.
    float *const part = p.part;
    const int64_t out_stride = part ? (int64_t)dim_z * 4 : p.out_stride[1] * (int64_t)sizeof(T);
    uint8_t *out = part ? reinterpret_cast<uint8_t *>(part_row(a, p, b, head, seg.from))
                        : reinterpret_cast<uint8_t *>(head_row<T>(p.out, p.out_stride, b, seg.from, head));
    out += (reverse ? (int64_t)max(len - C, 0) + C - 1 - c : (int64_t)c) * out_stride;
    const int64_t out_step = reverse ? -C * out_stride : C * out_stride;
    float16v o;
    const auto put = [&](int k) {
        const int short_by = C - rows_of_run(k);
        uint8_t *row = out;
        if (short_by > 0) { // the last run: it ends with the tile, backward in time at row 0
            row += reverse ? (k > 0 ? short_by * out_stride : 0) : -short_by * out_stride;
            if (c < short_by)
                return;
        }
        if (part)
            put_column<float, VEC>(reinterpret_cast<float *>(row), o, 1.0f, w, h, dim_z);
        else
            put_column<T, VEC>(reinterpret_cast<T *>(row), o, 1.0f, w, h, dim_z);
        out += out_step;
    };

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
        if (k > 0)
            put(k - 1);

        // scores, and x M with the state split into operands (in half precision times a power of two of each column,
        // which is what o's rows are multiplied back by)
        float16v s;
        float lift = 1.0f; // of this lane's column of the state
        if constexpr (kLifts<T>) {
            float top = 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = fmaxf(top, finite_size(m[d][i]));
            lift = lift_of(pair_max(top));
            if (h == 0)
                backs[c] = inverse_lift(lift);
            wave_fence();
        }
        for (bool careful = false;; careful = true) {
            s = zero16();
            o = zero16();
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                asm("" : "+v"(m[d])); // its parts are formed here, not kept from turn to turn
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const FragV<T> xf = TileT::row_frag(xt, c, 2 * d + half, h);
                    s = mma(TileT::row_frag(yt, c, 2 * d + half, h), xf, s);
                    FragV<T> mf[FEW];
                    split_half<T, FEW>(m[d], half, lift, mf, careful);
#pragma unroll
                    for (int n = 0; n < FEW; ++n)
                        o = mma(mf[n], xf, o);
                }
            }
            settle<T>();
            // an infinity of the state in parts is NaN
            if (FEW == 1 || careful || !__any(any_odd(o)))
                break;
        }
        FragV<T> zf[2];
        columns<T, TileT>(zf, zt, w, lane);
        const bool odd = __any(odd_values<T>(zf[0]) || odd_values<T>(zf[1]));

        if (n < C) { // rows before a short run are no tokens: 0 times an infinity is not theirs
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = acc_row(i, h) < C - n ? 0.0f : s[i];
        }
        float top = 0.0f;
        const float f = n < C ? g[max(c - (C - n), 0) + (reverse ? 0 : 1)] * p.read : come;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // a later token's score counts for nothing, whatever it is
            s[i] = acc_row(i, h) <= c ? s[i] * weight[i] : 0.0f;
            if constexpr (kLifts<T>)
                top = fmaxf(top, finite_size(s[i]));
        }
        const bool odd_scores = FEW > 1 && __any(any_odd(s));
        float score_lift = 1.0f;
        if constexpr (kLifts<T>) {
            score_lift = lift_of(pair_max(top));
            const Factors back(backs, h);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = o[i] * back.f[i >> 3][i & 7] * f;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] *= f;
        }
        bool careful = false;
        if (odd) { // what is NaN as it is needs no care: a step that overflowed is NaN nearly everywhere
            for (int i = 0; i < 16; ++i)
                careful |= o[i] == o[i] && 32 * w + acc_row(i, h) < dim_z;
            careful = __any(careful && c >= C - n);
        }
        FragV<T> fine[2] = {zf[0], zf[1]};
        if (careful) {
            // a later token's NaN times its score of 0 would be NaN here: what is not finite is left out of the
            // product and added where it is seen
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    fine[half][e] = not_finite((float)zf[half][e]) ? (T)0.0f : zf[half][e];
            for (int j = C - n; j < C; ++j) {
                // the score of token j and this lane's, from the lane and register that hold it
                const int from = (j >> 2) & 1, i0 = 4 * (j >> 3) + (j & 3);
                float score = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    score = i == i0 ? s[i] : score;
                score = __shfl(score, c + 32 * from);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float v = tile_value<T, C, DT>(zt, j, 32 * w + acc_row(i, h));
                    if (j <= c && not_finite(v))
                        o[i] += score * v;
                }
            }
        }
        // in half precision apart from o, so no power of two of one has to fit the other
        float16v seen = kLifts<T> ? zero16() : o;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            FragV<T> sf[FEW];
            split_half<T, FEW>(s, half, score_lift, sf, odd_scores);
#pragma unroll
            for (int n = 0; n < FEW; ++n)
                seen = mma(fine[half], sf[n], seen); // settled with the state
        }

        // the state behind the run
        decay(m, n < C ? g[n] : step.at(k));
        add_outer<T, TileT>(m, yt, Taken<T, PARTS>(zf, Factors(factors, h), odd || log_decay > 0.0f), lane);
        if constexpr (kLifts<T>) {
            const float back = inverse_lift(score_lift);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = fmaf(seen[i], back, o[i]);
        } else {
            o = seen;
        }
    }

    if (works && runs > 0)
        put(runs - 1);
    if (col >= dim_z)
        return;
    // rows behind the last token
    for (int row = seg.from + len + h; row < seg.to; row += 2) {
        if (p.part)
            part_row(a, p, b, head, row)[col] = 0.0f;
        else
            head_row<T>(p.out, p.out_stride, b, row, head)[col] = (T)0.0f;
    }
    if (p.last) { // the tokens are one segment
        float *last = p.last + b * p.last_stride[0] + head * p.last_stride[1] + col * p.last_stride[3];
        each_row_of_state<ND>(p.dim_x, h, [&](int d, int i, int row) { last[row * p.last_stride[2]] = m[d][i]; });
    }
}

// ---- what segments add to the state ---------------------------------------------
//
// M alone, from 0: no scores, no outputs.  Writing the states bounds it as much as its runs do.  Measured, bfloat16: 16
// heads of 128, 8160 tokens 31 us for one state a segment, 38 for the two gradients; 2 x 16 heads of 64 18 us.
template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(2 * DT, DT <= 64 ? 3 : 2) void linear_states(LinearArgs a)
{
    using G = Runs<T, DT, VEC, 2>;
    using RunT = typename G::RunT;
    using TileT = typename G::TileT;
    constexpr int ND = G::kBlocks, C = kRun;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t at = xcd_order(blockIdx.x, a.blocks);
    if (at >= a.blocks)
        return;
    const Work work(a.first + at, a.jobs, a.segments, a.heads);
    const LinearJob &p = a.job[work.job];
    const int b = work.b, head = work.head;
    const int t = (int)threadIdx.x, lane = t & 63, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const bool reverse = p.reverse != 0, works = 32 * w < p.dim_z;
    const Segment seg(a.lengths, b, (int)a.tokens, a.each, work.segment);
    if (!p.last && (reverse ? work.segment == 0 : work.segment == a.segments - 1))
        return; // no one asks what is behind it
    const int len = seg.len, runs = (len + C - 1) / C;

    const auto tile = [&](int buffer, int which) { return lds + (2 * buffer + which) * G::kTileBytes; };
    RunT ry(head_row<T>(p.y, p.y_stride, b, seg.from, head / p.y_share), p.y_stride[1], p.dim_x, reverse, len, t);
    RunT rz(head_row<T>(p.z, p.z_stride, b, seg.from, head / p.z_share), p.z_stride[1], p.dim_z, reverse, len, t);
    const auto rows_of_run = [&](int k) { return min(C, len - k * C); };
    const auto fetch = [&](int k, int buffer) {
        ry.fetch(tile(buffer, 0), rows_of_run(k), t);
        rz.fetch(tile(buffer, 1), rows_of_run(k), t);
    };
    if (runs > 0)
        fetch(0, 0);
    for (int i = 0; i < 4; ++i) // what no load writes
        RunT::StageT::clear(lds + i * G::kTileBytes, i % 2 == 1 ? p.dim_z : p.dim_x, t);
    float16v m[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
        m[d] = zero16();
    Powers g{reinterpret_cast<float *>(lds + G::kPowers)};
    float *factors = reinterpret_cast<float *>(lds + G::kFactors);
    const float log_decay = a.log_decay[head];
    g.fill(log_decay, C, t, G::kThreads);
    const Step step(log_decay, C);
    __syncthreads();
    if (t < C)
        factors[t] = g[C - 1 - t + (reverse ? 1 : 0)] * p.write;
    for (int k = 0; k < runs; ++k) {
        const int n = rows_of_run(k), buffer = k & 1;
        uint8_t *yt = tile(buffer, 0), *zt = tile(buffer, 1);
        ry.store(yt, n, t);
        rz.store(zt, n, t);
        __syncthreads();
        if (k + 1 < runs)
            fetch(k + 1, buffer ^ 1);
        if (!works)
            continue;
        FragV<T> zf[2];
        columns<T, TileT>(zf, zt, w, lane);
        const bool odd = __any(odd_values<T>(zf[0]) || odd_values<T>(zf[1]));
        decay(m, n < C ? g[n] : step.at(k));
        add_outer<T, TileT>(m, yt, Taken<T, kParts<T>>(zf, Factors(factors, h), odd || log_decay > 0.0f), lane);
    }
    StateImage<ND>::store(m, start_of(a, p, work.line, work.segment), w, lane);
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
// All of these are sums over tokens of an exact operand and one that is split in parts, so nothing is rounded to
// 16 bits on its way.  (bfloat16: three parts, as all states that leave a call; two would be off by up to 2^-17 of a term
// and save a few percent, with heads of 128, whose registers spill a little, 45 of 122 us.)  A segment begins with T = 0 and
// counts the steps within it; <T, dS> at its end, dS the gradient of the state there, counts them for the tokens
// behind it.  Its products and powers bound it (T and S are twice a state's registers, so two waves a SIMD is all there is): 16
// heads of 128, 8160 tokens 122 us; 32 x 6 heads of 32, 256 tokens, float16 11.
struct DecayArgs {
    const void *q, *k, *v, *dout;
    const float *state, *dstate;   // one segment: the call's
    const float *starts, *ends;    // else of each segment, [batch][head][segment]
    double *sums;                  // [batch][heads][segments]
    int64_t q_stride[3], k_stride[3], v_stride[3], dout_stride[3], state_stride[3], dstate_stride[3];
    const float *log_decay;
    const int32_t *lengths;
    int64_t tokens;
    int32_t batch, heads, share, dim, value_dim;
    int32_t segments, each, start_floats;
    float scale;
    uint32_t blocks, first;
};

// Waves that share 32 columns, each with its part of the states' rows: two waves a SIMD hide more than one.
template <int DT>
constexpr int kDecayWaves = DT == 64 || DT == 128 ? 2 : 1;

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(2 * DT * kDecayWaves<DT>, DT == 128 ? 2 : 1) void linear_decay(DecayArgs a)
{
    using G = Runs<T, DT, VEC, 4, kDecayWaves<DT>>;
    using RunT = typename G::RunT;
    using TileT = typename G::TileT;
    constexpr int ND = G::kBlocks, C = kRun, WAVES = kDecayWaves<DT>, MINE = ND / WAVES;
    constexpr int PARTS = kParts<T>;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t at = xcd_order(blockIdx.x, a.blocks);
    if (at >= a.blocks)
        return;
    const Work work(a.first + at, 1, a.segments, a.heads);
    const int b = work.b, head = work.head, kv = head / a.share;
    const int t = (int)threadIdx.x, lane = t & 63, c = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6), w = wave % ND, d0 = wave / ND * MINE, col = 32 * w + c;
    const Segment seg(a.lengths, b, (int)a.tokens, a.each, work.segment);
    const int len = seg.len, runs = (len + C - 1) / C;
    const int dims[4] = {a.dim, a.dim, a.value_dim, a.value_dim};

    const auto tile = [&](int buffer, int which) { return lds + (4 * buffer + which) * G::kTileBytes; };
    RunT run[4] = {
        RunT(head_row<T>(a.q, a.q_stride, b, seg.from, head), a.q_stride[1], a.dim, false, len, t),
        RunT(head_row<T>(a.k, a.k_stride, b, seg.from, kv), a.k_stride[1], a.dim, false, len, t),
        RunT(head_row<T>(a.v, a.v_stride, b, seg.from, kv), a.v_stride[1], a.value_dim, false, len, t),
        RunT(head_row<T>(a.dout, a.dout_stride, b, seg.from, head), a.dout_stride[1], a.value_dim, false, len, t)};
    const auto rows_of_run = [&](int k) { return min(C, len - k * C); };
    const auto fetch = [&](int k, int buffer) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            run[i].fetch(tile(buffer, i), rows_of_run(k), t);
    };
    if (runs > 0)
        fetch(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) // what no load writes
        RunT::StageT::clear(lds + i * G::kTileBytes, dims[i % 4], t);
    // this wave's rows of a state: of the call's, or of a segment's
    const int64_t place = (work.line * a.segments + work.segment) * a.start_floats;
    const auto each_mine = [&](const float *state, const int64_t *stride, const float *image, auto &&f) {
        if (a.segments > 1) {
#pragma unroll
            for (int d = 0; d < MINE; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    f(d, i, image[place + 4 * StateImage<ND>::at(d0 + d, i >> 2, w, lane) + (i & 3)]);
        } else if (state && col < a.value_dim) {
            const float *mine = state + b * stride[0] + head * stride[1] + col;
#pragma unroll
            for (int d = 0; d < MINE; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = 32 * (d0 + d) + state_row(acc_row(i, h));
                    if (row < a.dim)
                        f(d, i, mine[row * stride[2]]);
                }
        }
    };
    float16v s[MINE], u[MINE];
#pragma unroll
    for (int d = 0; d < MINE; ++d)
        s[d] = u[d] = zero16();
    each_mine(a.state, a.state_stride, a.starts, [&](int d, int i, float v) { s[d][i] = v; });
    // factors of a token: where a state takes it in for T and S, and for U and V, whose first token of a run
    // of n is token C - n of the tile
    Powers g{reinterpret_cast<float *>(lds + G::kPowers)};
    float *factors = reinterpret_cast<float *>(lds + G::kFactors);
    const float log_decay = a.log_decay[head];
    const bool grows = log_decay > 0.0f;
    g.fill(log_decay, C, t, G::kThreads);
    const Step decays(log_decay, C);
    const auto fill = [&](int n) {
        if (t < C) {
            const int i = max(t - (C - n), 0) + 1;
            factors[t] = a.scale * g[i];
            factors[C + t] = a.scale * (float)i * g[i];
            factors[2 * C + t] = (float)(C - 1 - t) * g[C - 1 - t];
            factors[3 * C + t] = g[C - 1 - t];
        }
    };
    __syncthreads();
    fill(C);
    float *steps = reinterpret_cast<float *>(lds + G::kSteps) + C;
    for (int e = t - C; e < C + 4; e += G::kThreads)
        steps[e] = e > 0 && e < C ? a.scale * (float)e * g[e] : 0.0f;
    double sum = 0.0; // of the runs' sums in 32 bits
    for (int k = 0; k < runs; ++k) {
        const int n = rows_of_run(k), buffer = k & 1;
        const uint8_t *qt = tile(buffer, 0), *kt = tile(buffer, 1), *vt = tile(buffer, 2), *dt = tile(buffer, 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            run[i].store(tile(buffer, i), n, t);
        if (n < C) {
            __syncthreads(); // the last run's factors
            fill(n);
        }
        __syncthreads();
        if (k + 1 < runs)
            fetch(k + 1, buffer ^ 1);
        if (k % (ND * WAVES) == wave) { // pairs within the run: the waves take turns
            float16v x = zero16(), y = zero16();
#pragma unroll
            for (int kk = 0; kk < 2 * ND; ++kk) {
                x = mma(TileT::row_frag(kt, c, kk, h), TileT::row_frag(qt, c, kk, h), x);
                y = mma(TileT::row_frag(vt, c, kk, h), TileT::row_frag(dt, c, kk, h), y);
            }
            settle<T>();
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = c - acc_row(i, h);
                part = fmaf(e > 0 ? x[i] * y[i] : 0.0f, steps[e], part);
            }
            sum += part;
        }
        if (32 * w >= a.value_dim)
            continue;
        const float whole = n < C ? g[n] : decays.at(k);
        float part = 0.0f;
        {
            FragV<T> zf[2];
            columns<T, TileT>(zf, dt, w, lane);
            const bool odd = __any(odd_values<T>(zf[0]) || odd_values<T>(zf[1])) || grows;
            const Taken<T, PARTS> for_u(zf, Factors(factors, h), odd), for_v(zf, Factors(factors + C, h), odd);
#pragma unroll
            for (int d = 0; d < MINE; ++d) {
                const FragV<T> yf[2] = {state_columns<T, TileT>(qt, 0, d0 + d, lane),
                                        state_columns<T, TileT>(qt, 16, d0 + d, lane)};
                const float16v x = for_u.times(yf, zero16()), y = for_v.times(yf, zero16());
                settle<T>();
                float by_t = 0.0f, by_s = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    by_t = fmaf(x[i], u[d][i], by_t);
                    by_s = fmaf(y[i], s[d][i], by_s);
                    u[d][i] = fmaf((float)n, s[d][i], u[d][i]) * whole;
                    s[d][i] *= whole;
                }
                part = fmaf(by_t, for_u.back, fmaf(by_s, for_v.back, part));
            }
        }
        FragV<T> zf[2];
        columns<T, TileT>(zf, vt, w, lane);
        const bool odd = __any(odd_values<T>(zf[0]) || odd_values<T>(zf[1])) || grows;
        const Taken<T, PARTS> to_t(zf, Factors(factors + 2 * C, h), odd), to_s(zf, Factors(factors + 3 * C, h), odd);
#pragma unroll
        for (int d = 0; d < MINE; ++d) {
            const FragV<T> yf[2] = {state_columns<T, TileT>(kt, 0, d0 + d, lane),
                                    state_columns<T, TileT>(kt, 16, d0 + d, lane)};
            if constexpr (kLifts<T>) {
                const float16v x = to_t.times(yf, zero16()), y = to_s.times(yf, zero16());
                settle<T>();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    u[d][i] = fmaf(x[i], to_t.back, u[d][i]);
                    s[d][i] = fmaf(y[i], to_s.back, s[d][i]);
                }
            } else {
                u[d] = to_t.times(yf, u[d]);
                s[d] = to_s.times(yf, s[d]);
            }
        }
        settle<T>();
        sum += part;
    }
    float part = 0.0f;
    each_mine(a.dstate, a.dstate_stride, a.ends, [&](int d, int i, float v) { part = fmaf(u[d][i], v, part); });
    sum += part;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        sum += __shfl_xor(sum, d);
    double *waves = reinterpret_cast<double *>(lds); // the tiles are done with
    __syncthreads();
    if (lane == 0)
        waves[wave] = sum;
    __syncthreads();
    if (t == 0) {
        for (int i = 1; i < ND * WAVES; ++i)
            sum += waves[i];
        a.sums[work.line * a.segments + work.segment] = sum;
    }
}

// Per element type; defined in one translation unit each (layers_linear_<type>.hip).
template <typename T>
struct Linear {
    static int sweep(LinearArgs a, bool vec, hipStream_t s);
    static int states(LinearArgs a, bool vec, hipStream_t s);
    static int decay(DecayArgs a, bool vec, hipStream_t s);
};

}  // namespace lic
