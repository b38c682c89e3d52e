// layers_attention_forward.hpp -- attention's forward kernels (included by the
// translation unit of each element type).
//
// One pass over the keys with a running maximum m and sum l of each row.  The
// maximum is only raised when a tile exceeds it by more than 2^8: below that the
// probabilities stay under 256, which 32-bit sums and both 16-bit types hold, and the
// accumulators need no scaling in most tiles.
#pragma once

#include "layers_attention.hpp"

namespace lic {
namespace {

constexpr float kSlack = 8.0f; // in powers of two

// Scores of one accumulator (keys along its rows) that a query does not see become -inf.  inside: all
// of them are within the query's range.
__device__ __forceinline__ void hide(float16v &s, const AttnArgs &a, const Range &range, bool inside,
                                     const uint8_t *mask, int key0, int h)
{
    if (mask)
        each_shown(mask, a.p.mask_stride[3], (int)a.p.keys, key0, h,
                   [&](int i, bool shown) { s[i] = shown ? s[i] : -INFINITY; });
    if (!inside) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = range.holds(key0 + acc_row(i, h)) ? s[i] : -INFINITY;
    }
}

// The running softmax of a lane's query over N accumulators of scores, which become
// probabilities relative to the running maximum.
template <int N, int ACC>
__device__ __forceinline__ void soften(float16v (&s)[N], float scale, float &m, float &l, float16v (&o)[ACC])
{
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, s[n][i]);
    top = pair_max(top) * scale;
    if (__builtin_amdgcn_ballot_w64(top > m + kSlack)) {
        const float next = fmaxf(m, top);
        const float shrink = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next);
        m = next;
        l *= shrink;
#pragma unroll
        for (int n = 0; n < ACC; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[n][i] *= shrink;
    }
    const float base = m == -INFINITY ? 0.0f : m; // nothing seen yet: exp(-inf) below
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], scale, -base));
            sum += s[n][i];
        }
    l += sum;
}

// A row that came out not finite, again and with the keys that it sees alone: a NaN or
// an infinity of a key it does not see is multiplied by its probability 0 above.
// Lane l takes key l of each 64, then column l (and l + 64) of the sum.
template <typename T>
__device__ void careful_row(const AttnArgs &a, int b, int head, int query, int len, int lo, int hi, float &m,
                            float &l, float (&o)[2])
{
    const int lane = threadIdx.x & 63, dim = (int)a.p.dim, kv = head / a.group;
    const Range range = keys_of(a, len, query);
    const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
    const uint8_t *mask = a.p.mask ? mask_row(a, b, head, query) : nullptr;
    m = -INFINITY, l = 0.0f, o[0] = o[1] = 0.0f;
    for (int k0 = lo; k0 < hi; k0 += 64) {
        const int key = k0 + lane;
        const bool seen = key < hi && range.holds(key) && (!mask || mask[key * a.p.mask_stride[3]] != 0);
        float s = -INFINITY;
        if (seen) {
            const T *k = head_row<T>(a.p.k, a.p.k_stride, b, key, kv);
            float dot = 0.0f;
            for (int d = 0; d < dim; ++d)
                dot = fmaf(up(q[d]), up(k[d]), dot);
            s = dot * a.scale_log2;
        }
        float top = s;
        for (int x = 32; x > 0; x >>= 1)
            top = fmaxf(top, __shfl_xor(top, x));
        const float next = fmaxf(m, top);
        const float shrink = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next);
        const float p = seen ? __builtin_amdgcn_exp2f(s - (next == -INFINITY ? 0.0f : next)) : 0.0f;
        m = next;
        float sum = p;
        for (int x = 32; x > 0; x >>= 1)
            sum += __shfl_xor(sum, x);
        l = l * shrink + sum;
        o[0] *= shrink, o[1] *= shrink;
        for (uint64_t left = __builtin_amdgcn_ballot_w64(seen); left; left &= left - 1) {
            const int j = __builtin_ctzll(left);
            const float pj = __shfl(p, j);
            const T *v = head_row<T>(a.p.v, a.p.v_stride, b, k0 + j, kv);
            if (lane < dim)
                o[0] = fmaf(pj, up(v[lane]), o[0]);
            if (lane + 64 < dim)
                o[1] = fmaf(pj, up(v[lane + 64]), o[1]);
        }
    }
}

__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---- many queries ----------------------------------------------------------
//
// A block of four waves holds 128 queries of one head, 32 a wave, in registers; keys
// and values pass through LDS in tiles of 64, two buffers, so one barrier a tile.
// A key tile serves four waves and costs each 1 LDS byte per 2 dim flops.
template <typename T, int DT, bool VEC>
struct TilesForward {
    static constexpr int kKeys = 64;
    using TileT = Tile<T, kKeys, DT>;
    using StageT = Stage<T, kKeys, DT, 256, VEC>;
    static constexpr int kLds = 4 * TileT::kBytes;
};

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(256, (DT <= 64 || sizeof(T) == 2) ? 2 : 1) void attention_tiles_forward(AttnArgs a)
{
    using G = TilesForward<T, DT, VEC>;
    using TileT = typename G::TileT;
    constexpr int KK = DT / 16, ND = DT / 32;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t block = xcd_order(blockIdx.x, a.blocks);
    if (block >= a.blocks)
        return;
    const uint32_t q_blocks = (uint32_t)((a.p.queries + 127) / 128);
    const uint32_t bh = block / q_blocks;
    const int head = (int)(bh % (uint32_t)a.p.heads), b = (int)(bh / (uint32_t)a.p.heads);
    const int kv = head / a.group;
    // the last queries see the most keys: they start first
    const int q0 = (int)(q_blocks - 1 - block % q_blocks) * 128;

    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6, h = lane >> 5;
    const int query = q0 + wave * 32 + (lane & 31);
    const int dim = (int)a.p.dim, len = key_length(a, b);
    const Range range = keys_of(a, len, query);
    const uint8_t *mask = a.p.mask ? mask_row(a, b, head, min(query, (int)a.p.queries - 1)) : nullptr;

    FragV<T> qf[KK];
    {
        const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            qf[kk] = row_from_memory<T, VEC>(q, query < a.p.queries, kk, h, dim);
    }
    float16v o[ND];
#pragma unroll
    for (int n = 0; n < ND; ++n)
        o[n] = zero16();
    float m = -INFINITY, l = 0.0f;

    int lo, hi;
    key_range(a, len, q0, min(q0 + 128, (int)a.p.queries), lo, hi);
    lo &= ~(G::kKeys - 1);
    const T *kbase = head_row<T>(a.p.k, a.p.k_stride, b, 0, kv);
    const T *vbase = head_row<T>(a.p.v, a.p.v_stride, b, 0, kv);
    const int64_t ks = a.p.k_stride[1], vs = a.p.v_stride[1];

    typename G::StageT kst, vst;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        G::StageT::clear(lds + i * TileT::kBytes, dim, t);
    const T *kp = kbase + lo * ks, *vp = vbase + lo * vs; // the next tile
    const auto fetch = [&](int buf, int rows) {
        kst.fetch(lds + buf * TileT::kBytes, kp, ks, rows, dim, t);
        vst.fetch(lds + (2 + buf) * TileT::kBytes, vp, vs, rows, dim, t);
        kp += ks * G::kKeys, vp += vs * G::kKeys;
    };
    const auto store = [&](int buf) {
        kst.store(lds + buf * TileT::kBytes, t);
        vst.store(lds + (2 + buf) * TileT::kBytes, t);
    };
    if (lo < hi) {
        fetch(0, len - lo);
        store(0);
    }
    loads_done();
    int buf = 0;
    for (int k0 = lo; k0 < hi; k0 += G::kKeys, buf ^= 1) {
        __syncthreads();
        const bool more = k0 + G::kKeys < hi;
        if (more)
            fetch(buf ^ 1, len - k0 - G::kKeys);
        if (!__all(range.misses(k0, G::kKeys))) {
            const uint8_t *kl = lds + buf * TileT::kBytes, *vl = lds + (2 + buf) * TileT::kBytes;
            float16v s[2] = {zero16(), zero16()};
            products_first();
            {
                Pipe<T, 2 * KK, 4> pipe;
                const auto read = [&](int i) {
                    return TileT::row_frag(kl, i / KK * 32 + (lane & 31), i % KK, h);
                };
                pipe.start(read);
                pipe.run(read, [&](int i, const FragV<T> &f) { s[i / KK] = mma(f, qf[i % KK], s[i / KK]); });
            }
            settle<T>();
            const auto read = [&](int i) { return TileT::col_frag(vl, i / ND * 16, i % ND, lane); };
            Pipe<T, 4 * ND, 4> pipe;
            pipe.start(read);
            const bool inside = __all(query >= a.p.queries || range.covers(k0, G::kKeys));
            if (mask || !inside) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    hide(s[n], a, range, inside, mask, k0 + n * 32, h);
            }
            products_over();
            soften(s, a.scale_log2, m, l, o);
            products_first();
            const FragV<T> p[4] = {operand<T>(s[0], 0), operand<T>(s[0], 1), operand<T>(s[1], 0),
                                   operand<T>(s[1], 1)};
            pipe.run(read, [&](int i, const FragV<T> &f) { o[i % ND] = mma(f, p[i / ND], o[i % ND]); });
        }
        if (more)
            store(buf ^ 1);
    }

    settle<T>();
    const float total = pair_sum(l);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    bool bad = false;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            bad |= not_finite(o[n][i]);
    uint64_t redo = rows_of(bad && query < a.p.queries);
    if (query < a.p.queries && !((redo >> (lane & 31)) & 1)) {
        T *out = head_row<T>(a.p.out, a.p.out_stride, b, query, head);
#pragma unroll
        for (int n = 0; n < ND; ++n)
            put_column<T, VEC>(out, o[n], inv, n, h, dim);
        if (h == 0)
            a.p.lse[((int64_t)b * a.p.heads + head) * a.p.queries + query] = log_sum(m, total);
    }
    for (; redo; redo &= redo - 1) {
        const AttnArgs &a = rare_args();
        const int qi = q0 + wave * 32 + __builtin_ctzll(redo);
        float cm, cl, co[2];
        careful_row<T>(a, b, head, qi, len, lo, hi, cm, cl, co);
        const float ci = cl == 0.0f ? 0.0f : 1.0f / cl;
        T *out = head_row<T>(a.p.out, a.p.out_stride, b, qi, head);
        if (lane < dim)
            out[lane] = down<T>(co[0] * ci);
        if (lane + 64 < dim)
            out[lane + 64] = down<T>(co[1] * ci);
        if (lane == 0)
            a.p.lse[((int64_t)b * a.p.heads + head) * a.p.queries + qi] = log_sum(cm, cl);
    }
}

// ---- few queries -------------------------------------------------------------
//
// The queries of all heads that share a kv head are packed into tiles of 32 rows
// (row r: query r / group, head r % group of them), so keys and values are read once
// for all of them; the key axis is split over blocks, and over a block's four waves,
// which take tiles of 32 keys in turn, each in its own LDS and with no barrier: the next
// tile is asked for before this one is waited for.  Memory bounds it: with a single row 31 of
// 32 columns of the products are idle, and the matrix units still need less time than the
// keys' way from HBM.  The waves' parts are joined in LDS, the blocks' by attention_rows_join.
template <typename T, int DT, bool VEC>
struct RowsForward {
    static constexpr int kKeys = 32;
    using TileT = Tile<T, kKeys, DT>;
    using StageT = Stage<T, kKeys, DT, 64, VEC>;
    static constexpr int kPair = 2 * TileT::kBytes;       // keys, values
    static constexpr int kBuffers = 8 * kPair <= 128 * 1024 ? 2 : 1;
    static constexpr int kSums = 32 * DT * 4;             // a wave's part at the end
    static constexpr int kRegion = kBuffers * kPair > kSums ? kBuffers * kPair : kSums;
    static constexpr int kLds = 4 * kRegion + 4 * 32 * 2 * 4;  // and m, l of each wave and row
};

// place of a sum: a row's columns rotated by four for each row, so that eight rows' four columns
// fall into different banks
template <int DT>
__device__ __forceinline__ int sum_at(int row, int d)
{
    return row * DT + (d + 4 * row) % DT;
}

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attention_rows_forward(AttnArgs a)
{
    using G = RowsForward<T, DT, VEC>;
    using TileT = typename G::TileT;
    constexpr int KK = DT / 16, ND = DT / 32, kRegion = G::kRegion;
    extern __shared__ __align__(16) uint8_t lds[];

    const int rows = (int)a.p.queries * a.group, row_tiles = (rows + 31) / 32;
    const uint32_t block = blockIdx.x;
    const int split = (int)(block % (uint32_t)a.splits);
    const uint32_t rest = block / (uint32_t)a.splits;
    const int row_tile = (int)(rest % (uint32_t)row_tiles);
    const uint32_t bk = rest / (uint32_t)row_tiles;
    const int kv = (int)(bk % (uint32_t)a.p.kv_heads), b = (int)(bk / (uint32_t)a.p.kv_heads);

    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6, h = lane >> 5;
    const int row = row_tile * 32 + (lane & 31);
    const int query = row / a.group, head = kv * a.group + row % a.group;
    const int dim = (int)a.p.dim, len = key_length(a, b);
    const Range range = keys_of(a, len, query);
    const uint8_t *mask = a.p.mask ? mask_row(a, b, head, min(query, (int)a.p.queries - 1)) : nullptr;

    FragV<T> qf[KK];
    {
        const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            qf[kk] = row_from_memory<T, VEC>(q, row < rows, kk, h, dim);
    }
    float16v o[ND];
#pragma unroll
    for (int n = 0; n < ND; ++n)
        o[n] = zero16();
    float m = -INFINITY, l = 0.0f;

    // this split's keys: an even share in whole tiles of the four waves
    int lo, hi;
    key_range(a, len, row_tile * 32 / a.group, min((row_tile * 32 + 31) / a.group + 1, (int)a.p.queries), lo, hi);
    const int share = ((hi - lo + a.splits - 1) / a.splits + 127) / 128 * 128;
    const int64_t first = (int64_t)lo + (int64_t)share * split;
    const int end = (int)least(hi, first + share);

    const T *kbase = head_row<T>(a.p.k, a.p.k_stride, b, 0, kv);
    const T *vbase = head_row<T>(a.p.v, a.p.v_stride, b, 0, kv);
    const int64_t ks = a.p.k_stride[1], vs = a.p.v_stride[1];
    uint8_t *mine = lds + wave * kRegion; // buffers of keys, values

    typename G::StageT kst, vst;
#pragma unroll
    for (int i = 0; i < 2 * G::kBuffers; ++i)
        G::StageT::clear(mine + i * TileT::kBytes, dim, lane);
    wave_fence();
    const auto fetch = [&](int64_t k, int buf) {
        kst.fetch(mine + buf * G::kPair, kbase + k * ks, ks, (int)(end - k), dim, lane);
        vst.fetch(mine + buf * G::kPair + TileT::kBytes, vbase + k * vs, vs, (int)(end - k), dim, lane);
    };
    loads_done();
    int64_t k0 = first + __builtin_amdgcn_readfirstlane(wave) * 32;
    int buf = 0;
    if (VEC && G::kBuffers == 2 && k0 < end)
        fetch(k0, 0);
    for (; k0 < end; k0 += 128) {
        uint8_t *kl = mine + buf * G::kPair, *vl = kl + TileT::kBytes;
        wave_fence();
        if (VEC && G::kBuffers == 2) {
            if (k0 + 128 < end) {
                fetch(k0 + 128, buf ^ 1);
                loads_done_but<2 * G::StageT::kEach>();
            } else {
                loads_done();
            }
            buf ^= 1;
        } else {
            fetch(k0, 0);
            kst.store(kl, lane);
            vst.store(vl, lane);
        }
        wave_fence();
        float16v s[1] = {zero16()};
        {
            Pipe<T, KK, KK % 4 ? 2 : 4> pipe;
            const auto read = [&](int i) { return TileT::row_frag(kl, lane & 31, i, h); };
            pipe.start(read);
            pipe.run(read, [&](int i, const FragV<T> &f) { s[0] = mma(f, qf[i], s[0]); });
        }
        settle<T>();
        // the tile may pass the split's end: those keys are the next split's
        const bool whole = k0 + 32 <= end;
        const bool inside = __all(row >= rows || range.covers((int)k0, 32));
        if (mask || !whole || !inside) {
            hide(s[0], a, range, inside, mask, (int)k0, h);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + acc_row(i, h) >= end)
                        s[0][i] = -INFINITY;
            }
        }
        soften(s, a.scale_log2, m, l, o);
        const FragV<T> p[2] = {operand<T>(s[0], 0), operand<T>(s[0], 1)};
        const auto read = [&](int i) { return TileT::col_frag(vl, i / ND * 16, i % ND, lane); };
        Pipe<T, 2 * ND, ND == 3 ? 3 : ND == 1 ? 2 : 4> pipe;
        pipe.start(read);
        pipe.run(read, [&](int i, const FragV<T> &f) { o[i % ND] = mma(f, p[i / ND], o[i % ND]); });
    }

    // a wave's part: sums [32][DT], then m and l
    settle<T>();
    l = pair_sum(l);
    bool bad = false;
    float *sums = reinterpret_cast<float *>(lds + wave * kRegion);
    float2 *stats = reinterpret_cast<float2 *>(lds + 4 * kRegion);
    wave_fence();
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            bad |= not_finite(o[n][i]) || not_finite(o[n][i + 1]) || not_finite(o[n][i + 2]) || not_finite(o[n][i + 3]);
            *reinterpret_cast<float4 *>(sums + sum_at<DT>(lane & 31, n * 32 + acc_row(i, h))) =
                make_float4(o[n][i], o[n][i + 1], o[n][i + 2], o[n][i + 3]);
        }
    if (h == 0)
        stats[wave * 32 + lane] = make_float2(m, l);
    wave_fence();
    for (uint64_t redo = rows_of(bad && row < rows); redo; redo &= redo - 1) {
        const AttnArgs &a = rare_args();
        const int j = __builtin_ctzll(redo);
        const int r = row_tile * 32 + j;
        float cm = -INFINITY, cl = 0.0f, co[2] = {0.0f, 0.0f};
        // this wave's tiles, each joined to the ones before
        for (int64_t c0 = first + wave * 32; c0 < end; c0 += 128) {
            float tm, tl, to[2];
            careful_row<T>(a, b, kv * a.group + r % a.group, r / a.group, len, (int)c0,
                           (int)least(c0 + 32, end), tm, tl, to);
            const float next = fmaxf(cm, tm);
            if (next == -INFINITY && tl == 0.0f)
                continue;
            const float wc = cl == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(cm - next);
            const float wt = tl == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(tm - next);
            cl = cl * wc + tl * wt;
            co[0] = (cl == 0.0f ? 0.0f : co[0] * wc) + (tl == 0.0f ? 0.0f : to[0] * wt);
            co[1] = (cl == 0.0f ? 0.0f : co[1] * wc) + (tl == 0.0f ? 0.0f : to[1] * wt);
            cm = next;
        }
        if (lane < DT)
            sums[sum_at<DT>(j, lane)] = co[0];
        if (lane + 64 < DT)
            sums[sum_at<DT>(j, lane + 64)] = co[1];
        if (lane == 0)
            stats[wave * 32 + j] = make_float2(cm, cl);
    }
    __syncthreads();

    // (m, l) of the waves become their weights, and of the first wave's the row's own in `whole`
    __shared__ float2 whole[32];
    if (t < 32) {
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            top = fmaxf(top, stats[w * 32 + t].x);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 st = stats[w * 32 + t];
            // a wave that saw nothing has sums of 0 and no weight (a NaN has one)
            const float f = st.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(st.x - top);
            total += f * st.y;
            stats[w * 32 + t].x = f;
        }
        whole[t] = make_float2(top, total);
    }
    __syncthreads();
    const float *all = reinterpret_cast<const float *>(lds);
    const int64_t lines = a.p.batch * a.p.heads * a.p.queries;
    for (int e = t; e < 8 * DT; e += 256) { // 32 rows of DT / 4
        const int j = e / (DT / 4), d = e % (DT / 4) * 4, r = row_tile * 32 + j;
        if (r >= rows)
            break;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = stats[w * 32 + j].x;
            const float4 v = *reinterpret_cast<const float4 *>(all + w * (kRegion / 4) + sum_at<DT>(j, d));
            sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
        }
        const float top = whole[j].x, total = whole[j].y;
        const int qi = r / a.group, hd = kv * a.group + r - qi * a.group;
        const int64_t line = ((int64_t)b * a.p.heads + hd) * a.p.queries + qi;
        if (a.splits == 1) {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            T *out = head_row<T>(a.p.out, a.p.out_stride, b, qi, hd) + d;
            const float v[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
            if constexpr (VEC) {
                Vec<T, 4> w;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w.v[i] = down<T>(v[i]);
                if (d < dim)
                    *reinterpret_cast<Vec<T, 4> *>(out) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (d + i < dim)
                        out[i] = down<T>(v[i]);
            }
            if (d == 0)
                a.p.lse[line] = log_sum(top, total);
        } else {
            // sums [split][line][DT], then top and total [split][line]
            *reinterpret_cast<float4 *>(a.part + (split * lines + line) * DT + d) = sum;
            if (d == 0)
                reinterpret_cast<float2 *>(a.part + a.splits * lines * DT)[split * lines + line] =
                    make_float2(top, total);
        }
    }
}

// The splits' parts of each row joined, a wave a row: lane s weighs split s, then all splits'
// sums are read at once.
template <typename T, int DT>
__global__ __launch_bounds__(256) void attention_rows_join(AttnArgs a)
{
    const int64_t lines = a.p.batch * a.p.heads * a.p.queries;
    const int64_t line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (line >= lines)
        return;
    const int lane = threadIdx.x & 63;
    const float *part = a.part + line * DT;
    const int64_t step = lines * DT;
    float2 stat = make_float2(-INFINITY, 0.0f);
    if (lane < a.splits)
        stat = reinterpret_cast<const float2 *>(a.part + a.splits * step)[lane * lines + line];
    float top = stat.x;
    for (int x = 32; x > 0; x >>= 1)
        top = fmaxf(top, __shfl_xor(top, x));
    // a split that saw nothing has sums of 0 and no weight
    const float weight = stat.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(stat.x - top);
    float total = weight * stat.y;
    for (int x = 32; x > 0; x >>= 1)
        total += __shfl_xor(total, x);
    float sum[2] = {0.0f, 0.0f};
    const int d0 = min(lane, DT - 1), d1 = min(lane + 64, DT - 1);
    for (int s0 = 0; s0 < a.splits; s0 += 8) {
        float v[2][8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float *p = part + min(s0 + u, a.splits - 1) * step;
            v[0][u] = p[d0];
            v[1][u] = DT > 64 ? p[d1] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            // lanes past the splits have no weight
            const float f = __shfl(weight, min(s0 + u, 63));
            sum[0] = fmaf(f, s0 + u < a.splits ? v[0][u] : 0.0f, sum[0]);
            sum[1] = fmaf(f, s0 + u < a.splits ? v[1][u] : 0.0f, sum[1]);
        }
    }
    const int query = (int)(line % a.p.queries);
    const int64_t bh = line / a.p.queries;
    const int head = (int)(bh % a.p.heads), b = (int)(bh / a.p.heads);
    T *out = head_row<T>(a.p.out, a.p.out_stride, b, query, head);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (lane < a.p.dim)
        out[lane] = down<T>(sum[0] * inv);
    if (lane + 64 < a.p.dim)
        out[lane + 64] = down<T>(sum[1] * inv);
    if (lane == 0)
        a.p.lse[line] = log_sum(top, total);
}

// ---- host ----------------------------------------------------------------------

template <typename T, int DT, bool VEC>
int run_forward(AttnArgs a, hipStream_t s)
{
    if (few_rows(a.p)) {
        using G = RowsForward<T, DT, VEC>;
        static const bool once = (allow_lds(attention_rows_forward<T, DT, VEC>, G::kLds), true);
        (void)once;
        a.splits = row_splits(a.p);
        const int64_t rows = a.p.queries * a.group;
        const int64_t blocks = (rows + 31) / 32 * a.p.batch * a.p.kv_heads * a.splits;
        if (blocks > 0x7fffffff)
            return RANS_E_ARG;
        attention_rows_forward<T, DT, VEC><<<(uint32_t)blocks, 256, G::kLds, s>>>(a);
        if (a.splits > 1) {
            const int64_t lines = a.p.batch * a.p.heads * a.p.queries;
            attention_rows_join<T, DT><<<(uint32_t)((lines + 3) / 4), 256, 0, s>>>(a);
        }
        return launched();
    }
    using G = TilesForward<T, DT, VEC>;
    static const bool once = (allow_lds(attention_tiles_forward<T, DT, VEC>, G::kLds > kTwoBlocks ? G::kLds : kTwoBlocks), true);
    (void)once;
    const int64_t blocks = (a.p.queries + 127) / 128 * a.p.batch * a.p.heads;
    if (blocks > 0x7fffff00)
        return RANS_E_ARG;
    a.blocks = (uint32_t)blocks;
    // Where windows or causal order make blocks of very different length, more LDS than they need
    // keeps a third block off a CU: more blocks are then left to fill the gaps that the short ones
    // leave (8160 x 8160 causal, 16 heads of 32 on 4: 131 us with two at a time, 152 with three).
    const bool uneven = a.p.window_left >= 0 || a.p.window_right >= 0;
    const int lds = uneven && G::kLds < kTwoBlocks ? kTwoBlocks : G::kLds;
    attention_tiles_forward<T, DT, VEC><<<xcd_grid(a.blocks), 256, lds, s>>>(a);
    return launched();
}

}  // namespace
}  // namespace lic
