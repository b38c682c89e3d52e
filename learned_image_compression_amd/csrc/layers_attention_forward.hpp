// layers_attention_forward.hpp -- attention's forward kernels (included by the
// translation unit of each element type).
//
// One pass over the keys with a running maximum m and sum l of each row.  The
// maximum is only raised when a tile exceeds it by more than 2^8: below that the
// probabilities stay under 256, which 32-bit sums and both 16-bit types hold, and the
// accumulators need no scaling in most tiles.  float16 takes them 2^7 times as large: of 10^5 keys
// below one of e^14, each p lies among its last numbers, and their sum was off by 0.05 of itself.
//
// Rounding: probabilities pass to the second product in the inputs' type, like any operand; scores,
// sums and accumulators stay in 32 bits.  For bfloat16 that is 0.0016 of out in the mean, as much as rounding
// out itself (0.0023 together; in float16 0.0003); two operands a product would buy it back at half as
// many products again.
#pragma once

#include "layers_attention.hpp"

namespace lic {
namespace {

constexpr float kSlack = 8.0f; // in powers of two
template <typename T>
constexpr float kRaise = std::is_same<T, f16>::value ? 7.0f : 0.0f; // 2^(8 + 7) is below float16's end

// Scores of one accumulator (keys along its rows) that a query does not see become -inf.  inside: all
// of them are within the query's range.  words: the mask's, where they were asked for before.
template <Masked MASK>
__device__ __forceinline__ void hide(float16v &s, const AttnArgs &a, const Range &range, bool inside,
                                     const uint8_t *mask, MaskWords &words, int key0, int h)
{
    const auto show = [&](int i, bool shown) { s[i] = shown ? s[i] : -INFINITY; };
    if constexpr (MASK == Masked::ahead)
        words.each_shown((int)a.p.keys, key0, h, show);
    else if constexpr (MASK == Masked::here)
        each_shown(mask, a.p.mask_stride[3], (int)a.p.keys, key0, h, show);
    if (!inside) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = range.holds(key0 + acc_row(i, h)) ? s[i] : -INFINITY;
    }
}

// The running softmax of a lane's query over N accumulators of scores, which become
// probabilities relative to the running maximum (less kRaise, as all that follows from them: at the
// end it comes off m, which is what the sums are relative to).
template <typename T, int N, int ACC>
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
    const float base = (m == -INFINITY ? 0.0f : m) - kRaise<T>; // nothing seen yet: exp(-inf) below
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

// A row that came out not finite (see Again), again and with the keys that it sees alone: a NaN or
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

// Where a split leaves its part of a row: sums [split][line][DT], then top and total [split][line].
template <int DT>
struct Part {
    float *sums;
    float2 *stat;

    __device__ __forceinline__ Part(const AttnArgs &a, int split, int64_t line)
    {
        const int64_t lines = a.p.batch * a.p.heads * a.p.queries, at = split * lines + line;
        sums = a.part + at * DT;
        stat = reinterpret_cast<float2 *>(a.part + a.splits * lines * DT) + at;
    }
};

// ---- many queries ----------------------------------------------------------
//
// A block of four waves holds 128 queries of one head, 32 a wave, in registers; keys
// and values pass through LDS in tiles of 64, two buffers, so one barrier a tile.
// A key tile serves four waves and costs each 1 LDS byte per 2 dim flops.  Where that makes few or
// unequal blocks the key axis is split and attention_rows_join adds the parts.  What bounds it: the
// exponentials with heads of 32 (8160 x 8160, 8 heads, bfloat16: 125 us, 4.3e12 a second), with wider
// ones the products and what the exponentials leave exposed of them (heads of 64: 168 us, 0.81 PFLOP/s;
// of 128: 258 us, 1.06 PFLOP/s); in 32 bits the products (8 x 8 heads of 64, 2048 x 2048: 540 us, 127 TFLOP/s).
template <typename T, int DT, bool VEC>
struct TilesForward {
    static constexpr int kKeys = 64;
    using TileT = Tile<T, kKeys, DT>;
    using StageT = Stage<T, kKeys, DT, 256, VEC>;
    static constexpr int kLds = 4 * TileT::kBytes;
};

template <typename T, int DT, bool VEC, Masked MASK>
__global__ __launch_bounds__(256, (DT <= 64 || sizeof(T) == 2) ? 2 : 1) void attention_tiles_forward(AttnArgs a)
{
    using G = TilesForward<T, DT, VEC>;
    using TileT = typename G::TileT;
    constexpr int KK = DT / 16, ND = DT / 32;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t place = xcd_order(blockIdx.x, a.blocks), block = a.first + place;
    if (place >= a.blocks)
        return;
    const uint32_t q_blocks = (uint32_t)((a.p.queries + 127) / 128);
    const uint32_t rest = block / q_blocks, bh = rest / (uint32_t)a.splits;
    const int head = (int)(bh % (uint32_t)a.p.heads), b = (int)(bh / (uint32_t)a.p.heads);
    const int kv = head / a.group;
    // the last queries see the most keys: they start first
    const int q0 = (int)(q_blocks - 1 - block % q_blocks) * 128;

    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6, h = lane >> 5;
    const int query = q0 + wave * 32 + (lane & 31);
    const int dim = (int)a.p.dim, len = key_length(a, b);
    const Range range = keys_of(a, len, query);
    const uint8_t *mask = nullptr;
    if constexpr (MASK != Masked::none)
        mask = mask_row(a, b, head, min(query, (int)a.p.queries - 1));

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
    if (a.splits > 1) { // an even share of the tiles
        const int share = ((hi - lo + G::kKeys - 1) / G::kKeys + a.splits - 1) / a.splits * G::kKeys;
        lo += share * (int)(rest % (uint32_t)a.splits);
        hi = min(hi, lo + share);
    }
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
    MaskWords words[2];
    const auto ask = [&](int k) {
        if constexpr (MASK == Masked::ahead) {
            words[0].ask(mask, (int)a.p.keys, k, h);
            words[1].ask(mask, (int)a.p.keys, k + 32, h);
        }
    };
    if (lo < hi) {
        fetch(0, len - lo);
        ask(lo);
        store(0);
    }
    loads_done();
    int buf = 0;
    for (int k0 = lo; k0 < hi; k0 += G::kKeys, buf ^= 1) {
        __syncthreads();
        const bool more = k0 + G::kKeys < hi;
        if (more)
            fetch(buf ^ 1, len - k0 - G::kKeys);
        if (__all(range.misses(k0, G::kKeys))) {
            ask(k0 + G::kKeys);
        } else {
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
            if (MASK != Masked::none || !inside) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    hide<MASK>(s[n], a, range, inside, mask, words[n], k0 + n * 32, h);
            }
            ask(k0 + G::kKeys);
            products_over();
            soften<T>(s, a.scale_log2, m, l, o);
            products_first();
            const FragV<T> p[4] = {operand<T>(s[0], 0), operand<T>(s[0], 1), operand<T>(s[1], 0),
                                   operand<T>(s[1], 1)};
            pipe.run(read, [&](int i, const FragV<T> &f) { o[i % ND] = mma(f, p[i / ND], o[i % ND]); });
            if constexpr (!VEC) // rows on their way take registers, so the sums may be moved next
                settle<T>();
        }
        if (more)
            store(buf ^ 1);
        if (MASK == Masked::ahead)
            loads_done();
    }

    settle<T>();
    m -= kRaise<T>;
    const float total = pair_sum(l);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    bool bad = false;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            bad |= not_finite(o[n][i]);
    // a sum of NaN: the scores that the row sees, and all of it is NaN
    uint64_t redo = rows_of(bad && query < a.p.queries && total == total);
    if (redo) {
        const AttnArgs &a = rare_args();
        Again again(redo);
        const int64_t step = a.p.mask_stride[3];
        for (int k0 = lo; k0 < hi; k0 += G::kKeys) // the last tile repeats the last key
            again.look(
                k0, G::kKeys, MASK == Masked::none && range.covers(k0, G::kKeys),
                [&](int key) {
                    Kinds v;
                    v.add(vbase + min(key, len - 1) * vs, dim);
                    return v.all_nan ? 7u : v.odd ? 3u : 0u;
                },
                [&](int key) { return range.holds(key) && (MASK == Masked::none || mask[key * step] != 0); });
        redo = again.which();
    }
    if (query < a.p.queries && !((redo >> (lane & 31)) & 1)) {
        const int64_t line = ((int64_t)b * a.p.heads + head) * a.p.queries + query;
        if (a.splits == 1) {
            T *out = head_row<T>(a.p.out, a.p.out_stride, b, query, head);
#pragma unroll
            for (int n = 0; n < ND; ++n)
                put_column<T, VEC>(out, o[n], inv, n, h, dim);
            if (h == 0)
                a.p.lse[line] = log_sum(m, total);
        } else {
            const Part<DT> part(a, (int)(rest % (uint32_t)a.splits), line);
#pragma unroll
            for (int n = 0; n < ND; ++n)
                put_column<float, true>(part.sums, o[n], 1.0f, n, h, DT);
            if (h == 0)
                *part.stat = make_float2(m, total);
        }
    }
    for (; redo; redo &= redo - 1) {
        const AttnArgs &a = rare_args();
        const int qi = q0 + wave * 32 + __builtin_ctzll(redo);
        float cm, cl, co[2];
        careful_row<T>(a, b, head, qi, len, lo, hi, cm, cl, co);
        const int64_t line = ((int64_t)b * a.p.heads + head) * a.p.queries + qi;
        if (a.splits > 1) {
            const Part<DT> part(a, (int)(rest % (uint32_t)a.splits), line);
            if (lane < DT)
                part.sums[lane] = co[0];
            if (lane + 64 < DT)
                part.sums[lane + 64] = co[1];
            if (lane == 0)
                *part.stat = make_float2(cm, cl);
            continue;
        }
        const float ci = cl == 0.0f ? 0.0f : 1.0f / cl;
        T *out = head_row<T>(a.p.out, a.p.out_stride, b, qi, head);
        if (lane < dim)
            out[lane] = down_apart<T>(co[0] * ci);
        if (lane + 64 < dim)
            out[lane + 64] = down_apart<T>(co[1] * ci);
        if (lane == 0)
            a.p.lse[line] = log_sum(cm, cl);
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
// keys' way from HBM (16 x 1 query of 16 heads of 64 on 4, up to 8160 keys, bfloat16: 24.5 us and 4 us for the join,
// 4.6 TB/s of what is in use).  The waves' parts are joined in LDS, the blocks' by attention_rows_join.
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
    const uint32_t block = a.first + blockIdx.x;
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
            MaskWords words;
            if (mask)
                hide<Masked::here>(s[0], a, range, inside, mask, words, (int)k0, h);
            else
                hide<Masked::none>(s[0], a, range, inside, mask, words, (int)k0, h);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + acc_row(i, h) >= end)
                        s[0][i] = -INFINITY;
            }
        }
        soften<T>(s, a.scale_log2, m, l, o);
        const FragV<T> p[2] = {operand<T>(s[0], 0), operand<T>(s[0], 1)};
        const auto read = [&](int i) { return TileT::col_frag(vl, i / ND * 16, i % ND, lane); };
        Pipe<T, 2 * ND, ND == 3 ? 3 : ND == 1 ? 2 : 4> pipe;
        pipe.start(read);
        pipe.run(read, [&](int i, const FragV<T> &f) { o[i % ND] = mma(f, p[i / ND], o[i % ND]); });
    }

    // a wave's part: sums [32][DT], then m and l
    settle<T>();
    m -= kRaise<T>;
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
    uint64_t redo = rows_of(bad && row < rows && l == l); // as above, of this wave's tiles
    if (redo) {
        const AttnArgs &a = rare_args();
        Again again(redo);
        const int64_t step = a.p.mask_stride[3];
        for (int64_t c0 = first + __builtin_amdgcn_readfirstlane(wave) * 32; c0 < end; c0 += 128)
            again.look(
                (int)c0, 32, !mask && c0 + 32 <= end && range.covers((int)c0, 32),
                [&](int key) {
                    Kinds v;
                    v.add(vbase + min(key, end - 1) * vs, dim);
                    return v.all_nan ? 7u : v.odd ? 3u : 0u;
                },
                [&](int key) { return key < end && range.holds(key) && (!mask || mask[key * step] != 0); });
        redo = again.which();
    }
    for (; redo; redo &= redo - 1) {
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
                    w.v[i] = down_apart<T>(v[i]);
                if (d < dim)
                    *reinterpret_cast<Vec<T, 4> *>(out) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (d + i < dim)
                        out[i] = down_apart<T>(v[i]);
            }
            if (d == 0)
                a.p.lse[line] = log_sum(top, total);
        } else {
            const Part<DT> part(a, split, line);
            *reinterpret_cast<float4 *>(part.sums + d) = sum;
            if (d == 0)
                *part.stat = make_float2(top, total);
        }
    }
}

// The splits' parts of each row joined (256 rows of 64, 8 splits 4 us; 48960 rows of 64, 4 splits 11.5 us,
// 4.9 TB/s): four columns of a row a thread, eight splits' parts asked for
// at once; more than eight are shared out over `groups` neighbouring threads (a power of two), whose
// sums are then joined the same way.
template <int DT>
constexpr int kJoinColumns = DT == 96 ? 32 : DT / 4; // threads of a row, of one group

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__(256) void attention_rows_join(AttnArgs a, int groups)
{
    constexpr int COLS = kJoinColumns<DT>;
    const int64_t id = (((int64_t)a.first + blockIdx.x) * 256 + threadIdx.x) / COLS, line = id / groups;
    if (line >= a.p.batch * a.p.heads * a.p.queries) // all threads of a row, or none
        return;
    const int d = (int)(threadIdx.x % COLS) * 4, at = DT == 96 ? min(d, DT - 4) : d;
    float top = -INFINITY, total = 0.0f;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = (int)(id % groups) * 8; s0 < a.splits; s0 += 8 * groups) {
        float2 stat[8];
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const Part<DT> part(a, min(s0 + u, a.splits - 1), line);
            stat[u] = *part.stat;
            v[u] = *reinterpret_cast<const float4 *>(part.sums + at);
        }
        const float before = top;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            top = fmaxf(top, stat[u].x);
        // a split that saw nothing has sums of 0 and no weight (a NaN has one)
        const float keep = total == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(before - top);
        total *= keep;
        sum.x *= keep, sum.y *= keep, sum.z *= keep, sum.w *= keep;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool is = s0 + u < a.splits && stat[u].y != 0.0f;
            const float f = is ? __builtin_amdgcn_exp2f(stat[u].x - top) : 0.0f;
            if (is) {
                total += f * stat[u].y;
                sum.x += f * v[u].x, sum.y += f * v[u].y, sum.z += f * v[u].z, sum.w += f * v[u].w;
            }
        }
    }
    for (int x = COLS; x < COLS * groups; x <<= 1) {
        const float theirs = __shfl_xor(top, x), both = fmaxf(top, theirs);
        const float their_total = __shfl_xor(total, x);
        const float f = total == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(top - both);
        const float g = their_total == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(theirs - both);
        top = both;
        total = f * total + g * their_total;
        sum.x = f * sum.x + g * __shfl_xor(sum.x, x), sum.y = f * sum.y + g * __shfl_xor(sum.y, x);
        sum.z = f * sum.z + g * __shfl_xor(sum.z, x), sum.w = f * sum.w + g * __shfl_xor(sum.w, x);
    }
    if (id % groups != 0 || d >= DT)
        return;
    const int query = (int)(line % a.p.queries);
    const int64_t bh = line / a.p.queries;
    const int head = (int)(bh % a.p.heads), b = (int)(bh / a.p.heads), dim = (int)a.p.dim;
    T *out = head_row<T>(a.p.out, a.p.out_stride, b, query, head) + d;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    Vec<T, 4> w;
    w.v[0] = down_apart<T>(sum.x * inv), w.v[1] = down_apart<T>(sum.y * inv);
    w.v[2] = down_apart<T>(sum.z * inv), w.v[3] = down_apart<T>(sum.w * inv);
    if constexpr (VEC) {
        if (d < dim)
            *reinterpret_cast<Vec<T, 4> *>(out) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < dim)
                out[e] = w.v[e];
    }
    if (d == 0)
        a.p.lse[line] = log_sum(top, total);
}

// ---- host ----------------------------------------------------------------------

template <typename T, int DT, bool VEC>
int run_forward(AttnArgs a, hipStream_t s)
{
    const ForwardPlan plan = forward_plan(a.p);
    a.splits = plan.splits;
    const auto join = [&] {
        if (a.splits > 1) {
            const int64_t lines = a.p.batch * a.p.heads * a.p.queries;
            int groups = 1;
            while (8 * groups < a.splits && 2 * groups * kJoinColumns<DT> <= 64)
                groups *= 2;
            const int64_t threads = lines * groups * kJoinColumns<DT>;
            in_pieces((threads + 255) / 256, 256, [&](int64_t first, uint32_t blocks) {
                a.first = (uint32_t)first;
                attention_rows_join<T, DT, VEC><<<blocks, 256, 0, s>>>(a, groups);
            });
        }
    };
    if (plan.few) {
        using G = RowsForward<T, DT, VEC>;
        if (const int rc = allow_lds<attention_rows_forward<T, DT, VEC>>(G::kLds))
            return rc;
        const int64_t rows = a.p.queries * a.group;
        const int64_t blocks = (rows + 31) / 32 * a.p.batch * a.p.kv_heads * a.splits;
        if (blocks > kMostBlocks)
            return RANS_E_ARG;
        in_pieces(blocks, 256, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first;
            attention_rows_forward<T, DT, VEC><<<piece, 256, G::kLds, s>>>(a);
        });
        join();
        return launched();
    }
    using G = TilesForward<T, DT, VEC>;
    const int64_t blocks = (a.p.queries + 127) / 128 * a.p.batch * a.p.heads * a.splits;
    if (blocks > kMostBlocks)
        return RANS_E_ARG;
    // Where windows or causal order make blocks of very different length, more LDS than they need
    // keeps a third block off a CU: more blocks are then left to fill the gaps that the short ones
    // leave (8160 x 8160 causal, 16 heads of 32 on 4: 131 us with two at a time, 152 with three).
    const bool uneven = a.p.window_left >= 0 || a.p.window_right >= 0;
    const int lds = uneven && G::kLds < kTwoBlocks ? kTwoBlocks : G::kLds;
    const int rc = with_mask<VEC && (sizeof(T) == 2 ? DT <= 96 : DT != 64)>(a.p, [&](auto masked) {
        constexpr auto kernel = attention_tiles_forward<T, DT, VEC, decltype(masked)::value>;
        if (const int rc = allow_lds<kernel>(G::kLds > kTwoBlocks ? G::kLds : kTwoBlocks))
            return rc;
        in_pieces(blocks, 256, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first, a.blocks = piece;
            kernel<<<xcd_grid(piece), 256, lds, s>>>(a);
        });
        return (int)RANS_OK;
    });
    if (rc)
        return rc;
    join();
    return launched();
}

}  // namespace
}  // namespace lic
