// layers_attention_backward.hpp -- attention's backward kernels (included by the
// translation unit of each element type).
//
//   p_ij = exp(scale q_i . k_j - lse_i),  D_i = dout_i . out_i
//   dv_j = sum_i p_ij dout_i,  ds_ij = p_ij (dout_i . v_j - D_i)
//   dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// The probabilities are formed again rather than kept: two kernels walk the pairs, one with
// keys held (dk, dv) and one with queries held (dq), so every sum stays in the registers
// of one wave and no atomic decides an order.  That is seven products where five would do
// if one kernel's waves added into another's rows.
//
// Rounding: p and ds pass to their second product in the inputs' type, like any
// operand; sums, D and the scores stay in 32 bits.  For bfloat16 that is 0.0017 of dq and dk in
// the mean, as much as rounding the results themselves (0.0026 together; two operands a product
// would buy it back at twice the products).  p is rounded as 2^10 p, which costs
// nothing (the power goes into lse, its inverse into D and the last scaling): among
// thousands of keys most p lie below float16's normal numbers.  ds is smaller still, and as
// small as dout and v make it: in float16 a power of two of each row lifts it (Lift).
#pragma once

#include "layers_attention.hpp"

namespace lic {
namespace {

constexpr float kLift = 10.0f, kLower = 1.0f / 1024.0f; // 2^10 and its inverse

// The power of two, of a lane's row (a query, or a key), that ds takes on its way into float16.  It
// begins at 2^60 and comes down, the row's sums with it, wherever a ds exceeds 2^15 with it: the largest
// so far then lies at 2^8 to 2^15, what is 2^-22 of it or more keeps its precision, and nothing overflows.  (8160 keys, heads of 64, dout of size 1e-4: with ds as it is 45%
// of them are 0 and dq is off by 0.1 of itself.)  It takes 2 to 7% of a float16 training pass (32 x 6
// heads of 32, 256 x 256, with a mask 45.8 -> 46.8 us; 8 x 8 of 64, 510 x 510 causal 48.9 -> 52.2; 8160 x 8160
// causal, 16 heads of 128 on 4 1.28 -> 1.32 ms), most of it the product in the keys' kernel.
// bfloat16 and 32 bits need none.
template <typename T>
struct Lift {
    static constexpr bool kOn = std::is_same<T, f16>::value;
    static constexpr float kMost = 32768.0f;
    static constexpr int kAim = 8;
    float f = kOn ? 0x1p60f : 1.0f;

    // ds (f times its value) of 16 pairs, and the row's sums and what else f scales
    template <int ACC>
    __device__ __forceinline__ void fit(float16v &ds, float16v (&sums)[ACC], float *more, int count)
    {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, fabsf(ds[i]));
        if (__builtin_amdgcn_ballot_w64(top > kMost)) {
            top = 0.0f; // of the finite ones: the others stay as they are
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = fmaxf(top, not_finite(ds[i]) ? 0.0f : fabsf(ds[i]));
            top = pair_max(top); // a row's two lanes
            const float by = top > kMost ? __builtin_amdgcn_ldexpf(1.0f, kAim - __builtin_amdgcn_frexp_expf(top)) : 1.0f;
            f *= by;
            for (int i = 0; i < count; ++i)
                more[i] *= by;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ds[i] *= by;
#pragma unroll
            for (int n = 0; n < ACC; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sums[n][i] *= by;
        }
    }
    // the sums as they are
    template <int ACC>
    __device__ __forceinline__ void undo(float16v (&sums)[ACC]) const
    {
        const float by = 1.0f / f;
#pragma unroll
        for (int n = 0; n < ACC; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sums[n][i] *= by;
    }
};

// One query's gradient with the keys it sees alone (see careful_row of the forward call).
template <typename T>
__device__ void careful_dq(const AttnArgs &a, int b, int head, int query, int len, int lo, int hi, float lse,
                           float delta, float (&dq)[2])
{
    const int lane = threadIdx.x & 63, dim = (int)a.p.dim, kv = head / a.group;
    const Range range = keys_of(a, len, query);
    const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
    const T *g = head_row<T>(a.p.dout, a.p.dout_stride, b, query, head);
    const uint8_t *mask = a.p.mask ? mask_row(a, b, head, query) : nullptr;
    dq[0] = dq[1] = 0.0f;
    for (int k0 = lo; k0 < hi; k0 += 64) {
        const int key = k0 + lane;
        const bool seen = key < hi && range.holds(key) && (!mask || mask[key * a.p.mask_stride[3]] != 0);
        float ds = 0.0f;
        if (seen) {
            const T *k = head_row<T>(a.p.k, a.p.k_stride, b, key, kv);
            const T *v = head_row<T>(a.p.v, a.p.v_stride, b, key, kv);
            float s = 0.0f, dp = 0.0f;
            for (int d = 0; d < dim; ++d) {
                s = fmaf(up(q[d]), up(k[d]), s);
                dp = fmaf(up(g[d]), up(v[d]), dp);
            }
            ds = __builtin_amdgcn_exp2f(fmaf(s, a.scale_log2, -lse)) * fmaf(dp, kLower, -delta);
        }
        for (uint64_t left = __builtin_amdgcn_ballot_w64(seen); left; left &= left - 1) {
            const int j = __builtin_ctzll(left);
            const float x = __shfl(ds, j);
            const T *k = head_row<T>(a.p.k, a.p.k_stride, b, k0 + j, kv);
            if (lane < dim)
                dq[0] = fmaf(x, up(k[lane]), dq[0]);
            if (lane + 64 < dim)
                dq[1] = fmaf(x, up(k[lane + 64]), dq[1]);
        }
    }
}

// One key's gradients from the queries [lo, hi) of a head that see it alone, added to dk and (2^10
// times) dv.
template <typename T>
__device__ void careful_dkv(const AttnArgs &a, int b, int head, int key, int len, int lo, int hi, float (&dk)[2],
                            float (&dv)[2])
{
    const int lane = threadIdx.x & 63, dim = (int)a.p.dim, kv = head / a.group;
    const Range range = queries_of(a, len, key);
    const T *k = head_row<T>(a.p.k, a.p.k_stride, b, key, kv);
    const T *v = head_row<T>(a.p.v, a.p.v_stride, b, key, kv);
    const int64_t line0 = ((int64_t)b * a.p.heads + head) * a.p.queries;
    for (int q0 = lo; q0 < hi; q0 += 64) {
        const int query = q0 + lane;
        const bool seen = query < hi && range.holds(query) &&
                          (!a.p.mask || mask_row(a, b, head, query)[key * a.p.mask_stride[3]] != 0);
        float p = 0.0f, ds = 0.0f;
        if (seen) {
            const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
            const T *g = head_row<T>(a.p.dout, a.p.dout_stride, b, query, head);
            float s = 0.0f, dp = 0.0f;
            for (int d = 0; d < dim; ++d) {
                s = fmaf(up(q[d]), up(k[d]), s);
                dp = fmaf(up(g[d]), up(v[d]), dp);
            }
            p = __builtin_amdgcn_exp2f(fmaf(s, a.scale_log2, -a.row_lse[line0 + query]));
            ds = p * fmaf(dp, kLower, -a.row_delta[line0 + query]);
        }
        for (uint64_t left = __builtin_amdgcn_ballot_w64(seen); left; left &= left - 1) {
            const int j = __builtin_ctzll(left);
            const float pj = __shfl(p, j), dj = __shfl(ds, j);
            const T *q = head_row<T>(a.p.q, a.p.q_stride, b, q0 + j, head);
            const T *g = head_row<T>(a.p.dout, a.p.dout_stride, b, q0 + j, head);
            if (lane < dim) {
                dk[0] = fmaf(dj, up(q[lane]), dk[0]);
                dv[0] = fmaf(pj, up(g[lane]), dv[0]);
            }
            if (lane + 64 < dim) {
                dk[1] = fmaf(dj, up(q[lane + 64]), dk[1]);
                dv[1] = fmaf(pj, up(g[lane + 64]), dv[1]);
            }
        }
    }
}

// ---- dk, dv ------------------------------------------------------------------
//
// A block holds 128 keys of one kv head, 32 a wave; the queries of the heads that share it
// pass through LDS in tiles of 32 or 64 with their dout, lse and D.  Scores have queries along
// the accumulator's rows and keys across the lanes.
//
// Four waves hold their keys' and values' fragments in registers.  With heads of 128 in 16
// bits those and the accumulators (192 registers) leave no room for a second wave on
// a SIMD, and one wave cannot overlap its exponentials with its products.  There keys and
// values stay in LDS, half as many reads again, and eight waves work on a block: the upper
// four take the second half of each query tile and their sums are added at the end.
//
// Products bound it with wide heads: 8160 x 8160 causal, 16 heads of 128 on 4, bfloat16 590 to 625 us,
// 0.87 to 0.93 PFLOP/s of the four products (a large library product: 1.13).  32 x 6 heads of 32, 256 x 256,
// float16 with a mask 18 us: four tiles a block, so loads, the mask and the start of each block.
template <typename T, int DT>
struct KeysBackward {
    static constexpr bool kWide = sizeof(T) == 2 && DT == 128;
    static constexpr int kThreads = kWide ? 512 : 256;
    static constexpr int kQueries = sizeof(T) == 4 ? 32 : 64;
    using TileT = Tile<T, kQueries, DT>;
    using KeysT = Tile<T, 128, DT>;
    static constexpr int kKeys = 4 * TileT::kBytes;          // after two buffers of q and dout: keys, values
    static constexpr int kStats = kKeys + (kWide ? 2 * KeysT::kBytes : 0); // two buffers of lse, D
    static constexpr int kLds = kStats + 2 * 2 * kQueries * 4;
    static constexpr int kWaves = sizeof(T) == 2 || DT == 32 ? 2 : 1; // of a SIMD
};

template <typename T, int DT, bool VEC>
__global__ __launch_bounds__((KeysBackward<T, DT>::kThreads), (KeysBackward<T, DT>::kWaves)) void
attention_keys_backward(AttnArgs a)
{
    using G = KeysBackward<T, DT>;
    using TileT = typename G::TileT;
    constexpr int KK = DT / 16, ND = DT / 32, NQ = G::kQueries;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t place = xcd_order(blockIdx.x, a.blocks), block = a.first + place;
    if (place >= a.blocks)
        return;
    const uint32_t k_blocks = (uint32_t)((a.p.keys + 127) / 128);
    const int key0 = (int)(block % k_blocks) * 128; // the first keys are seen by the most queries
    const uint32_t rest = block / k_blocks;
    const int split = (int)(rest % (uint32_t)a.splits);
    const uint32_t bk = rest / (uint32_t)a.splits;
    const int kv = (int)(bk % (uint32_t)a.p.kv_heads), b = (int)(bk / (uint32_t)a.p.kv_heads);

    const int t = (int)threadIdx.x, lane = t & 63, wave = (t >> 6) & 3, upper = t >> 8, h = lane >> 5;
    const int key = key0 + wave * 32 + (lane & 31);
    const int dim = (int)a.p.dim, len = key_length(a, b);
    const Range range = queries_of(a, len, key);

    // fragments of the wave's keys and values: held, or read from LDS each time
    FragV<T> kf[G::kWide ? 1 : KK], vf[G::kWide ? 1 : KK];
    const uint8_t *kl = lds + G::kKeys, *vl = kl + G::KeysT::kBytes;
    if constexpr (G::kWide) {
        using WholeT = Stage<T, 128, DT, G::kThreads, VEC>;
        WholeT ks, vs;
        ks.clear(lds + G::kKeys, dim, t);
        vs.clear(lds + G::kKeys + G::KeysT::kBytes, dim, t);
        if (key0 < len) {
            ks.fetch(lds + G::kKeys, head_row<T>(a.p.k, a.p.k_stride, b, key0, kv), a.p.k_stride[1], len - key0, dim,
                     t);
            vs.fetch(lds + G::kKeys + G::KeysT::kBytes, head_row<T>(a.p.v, a.p.v_stride, b, key0, kv),
                     a.p.v_stride[1], len - key0, dim, t);
            ks.store(lds + G::kKeys, t);
            vs.store(lds + G::kKeys + G::KeysT::kBytes, t);
        }
    } else {
        const T *k = head_row<T>(a.p.k, a.p.k_stride, b, key, kv);
        const T *v = head_row<T>(a.p.v, a.p.v_stride, b, key, kv);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            kf[kk] = row_from_memory<T, VEC>(k, key < len, kk, h, dim);
            vf[kk] = row_from_memory<T, VEC>(v, key < len, kk, h, dim);
        }
    }
    float16v dk[ND], dv[ND];
#pragma unroll
    for (int n = 0; n < ND; ++n)
        dk[n] = dv[n] = zero16();
    Lift<T> lift; // of the lane's key

    // tiles of all heads in one row: this split takes an even share of them
    int lo = 0, hi = 0;
    if (key0 < len)
        query_range(a, len, key0, min(key0 + 128, len), lo, hi);
    lo &= ~(NQ - 1);
    const int tiles = (hi - lo + NQ - 1) / NQ, all = tiles * a.group;
    const int share = (all + a.splits - 1) / a.splits;
    const int first = min(all, split * share), end = min(all, first + share);

    using StageT = Stage<T, NQ, DT, G::kThreads, VEC>;
    StageT qst, gst;
    // the tile that is loaded next: its head, first query, and where its rows begin
    int head = kv * a.group + (tiles ? first / tiles : 0), q_next = lo + (tiles ? first % tiles : 0) * NQ;
    const int64_t qs = a.p.q_stride[1] * NQ, gs = a.p.dout_stride[1] * NQ;
    const T *qp = nullptr, *gp = nullptr;
    const float *lp = nullptr, *dp_row = nullptr;
    const auto enter = [&]() {
        qp = head_row<T>(a.p.q, a.p.q_stride, b, q_next, head);
        gp = head_row<T>(a.p.dout, a.p.dout_stride, b, q_next, head);
        const int64_t line = ((int64_t)b * a.p.heads + head) * a.p.queries + q_next;
        lp = a.row_lse + line;
        dp_row = a.row_delta + line;
    };
    const auto fetch = [&](int buf) {
        const int rows = (int)a.p.queries - q_next;
        qst.fetch(lds + buf * TileT::kBytes, qp, a.p.q_stride[1], rows, dim, t);
        gst.fetch(lds + (2 + buf) * TileT::kBytes, gp, a.p.dout_stride[1], rows, dim, t);
        // the first wave brings the tile's lse, the second its D
        const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + G::kStats +
                            buf * 2 * NQ * 4;
        const int turn = __builtin_amdgcn_readfirstlane(t >> 6);
        if (turn < 2 && lane < NQ)
            load_lds<4>(to + turn * NQ * 4, turn ? dp_row : lp, min(lane, rows - 1) * 4);
        q_next += NQ, qp += qs, gp += gs, lp += NQ, dp_row += NQ;
        if (q_next >= lo + tiles * NQ) {
            q_next = lo;
            ++head;
            if (head < (kv + 1) * a.group)
                enter();
        }
    };
    const auto store = [&](int buf) {
        qst.store(lds + buf * TileT::kBytes, t);
        gst.store(lds + (2 + buf) * TileT::kBytes, t);
        loads_done();
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
        StageT::clear(lds + i * TileT::kBytes, dim, t);
    int q_cur = q_next, head_cur = head; // the tile worked on
    if (first < end) {
        enter();
        fetch(0);
        store(0);
    }
    loads_done();
    int buf = 0;
    for (int i = first; i < end; ++i, buf ^= 1) {
        __syncthreads();
        const int q0 = q_cur, q_head = head_cur;
        if (i + 1 < end) {
            q_cur = q_next, head_cur = head;
            fetch(buf ^ 1);
        }
#pragma unroll
        for (int half_tile = 0; half_tile < (G::kWide ? 1 : NQ / 32); ++half_tile) {
            const int n32 = (G::kWide ? upper : half_tile) * 32;
            const int qn = q0 + n32;
            if (__all(range.misses(qn, 32)))
                continue;
            const uint8_t *ql = lds + buf * TileT::kBytes, *gl = lds + (2 + buf) * TileT::kBytes;
            const float *lse = reinterpret_cast<const float *>(lds + G::kStats) + buf * 2 * NQ + n32;
            const float *delta = lse + NQ;
            float16v s = zero16(), dp = zero16();
            products_first();
            if constexpr (G::kWide) {
                // q and keys in turn, then dout and values
                const auto read = [&](int i) {
                    const int kk = i / 2 % KK;
                    if (i % 2)
                        return G::KeysT::row_frag(i < 2 * KK ? kl : vl, wave * 32 + (lane & 31), kk, h);
                    return TileT::row_frag(i < 2 * KK ? ql : gl, n32 + (lane & 31), kk, h);
                };
                Pipe<T, 4 * KK, 4> pipe;
                FragV<T> left;
                pipe.start(read);
                pipe.run(read, [&](int i, const FragV<T> &f) {
                    if (i % 2 == 0)
                        left = f;
                    else if (i < 2 * KK)
                        s = mma(left, f, s);
                    else
                        dp = mma(left, f, dp);
                });
            } else {
                Pipe<T, 2 * KK, 4> pipe;
                const auto read = [&](int i) {
                    return TileT::row_frag(i < KK ? ql : gl, n32 + (lane & 31), i % KK, h);
                };
                pipe.start(read);
                pipe.run(read, [&](int i, const FragV<T> &f) {
                    if (i < KK)
                        s = mma(f, kf[G::kWide ? 0 : i % KK], s);
                    else
                        dp = mma(f, vf[G::kWide ? 0 : i % KK], dp);
                });
            }
            settle<T>();
            // operands of the second products: (half, dout then q, block of columns)
            const auto read = [&](int i) {
                return TileT::col_frag(i / ND % 2 ? ql : gl, n32 + i / (2 * ND) * 16, i % ND, lane);
            };
            Pipe<T, 4 * ND, 4> pipe;
            pipe.start(read);
            products_over();
            // lanes beyond the keys are not stored
            const bool inside = __all(key >= len || range.covers(qn, 32));
#pragma unroll
            for (int i4 = 0; i4 < 16; i4 += 4) {
                const float4 ls = *reinterpret_cast<const float4 *>(lse + acc_row(i4, h));
                const float4 de = *reinterpret_cast<const float4 *>(delta + acc_row(i4, h));
                const float l4[4] = {ls.x, ls.y, ls.z, ls.w}, d4[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = i4 + e;
                    s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale_log2, -l4[e]));
                    dp[r] = s[r] * fmaf(dp[r], kLower, -d4[e]);
                    if constexpr (Lift<T>::kOn)
                        dp[r] *= lift.f;
                }
            }
            const auto show = [&](int r, bool shown) {
                s[r] = shown ? s[r] : 0.0f;
                dp[r] = shown ? dp[r] : 0.0f;
            };
            if (a.p.mask)
                each_shown(mask_row(a, b, q_head, 0) + min(key, (int)a.p.keys - 1) * a.p.mask_stride[3],
                           a.p.mask_stride[2], (int)a.p.queries, qn, h, show);
            if (!inside) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    show(r, range.holds(qn + acc_row(r, h)));
            }
            if constexpr (Lift<T>::kOn)
                lift.fit(dp, dk, nullptr, 0);
            products_first();
            const FragV<T> p[2] = {operand<T>(s, 0), operand<T>(s, 1)};
            const FragV<T> ds[2] = {operand<T>(dp, 0), operand<T>(dp, 1)};
            pipe.run(read, [&](int i, const FragV<T> &f) {
                const int half = i / (2 * ND), n = i % ND;
                if (i / ND % 2)
                    dk[n] = mma(f, ds[half], dk[n]);
                else
                    dv[n] = mma(f, p[half], dv[n]);
            });
        }
        if (i + 1 < end)
            store(buf ^ 1);
    }

    settle<T>();
    if constexpr (Lift<T>::kOn)
        lift.undo(dk);
    if constexpr (G::kWide) {
        float *sums = reinterpret_cast<float *>(lds) + wave * (2 * ND * 16 * 64) + lane;
        __syncthreads();
        if (upper) {
#pragma unroll
            for (int n = 0; n < ND; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sums[(n * 16 + i) * 64] = dk[n][i];
                    sums[((ND + n) * 16 + i) * 64] = dv[n][i];
                }
        }
        __syncthreads();
        if (upper)
            return;
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                dk[n][i] += sums[(n * 16 + i) * 64];
                dv[n][i] += sums[((ND + n) * 16 + i) * 64];
            }
    }
    bool bad = false;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            bad |= not_finite(dk[n][i]) || not_finite(dv[n][i]);
    uint64_t redo = rows_of(bad && key < len);
    if (redo) {
        const AttnArgs &a = rare_args();
        Kinds own_key, own_value;
        if (key < len) {
            own_key.add(head_row<T>(a.p.k, a.p.k_stride, b, key, kv), dim);
            own_value.add(head_row<T>(a.p.v, a.p.v_stride, b, key, kv), dim);
        }
        const uint64_t nan_keys = rows_of(own_key.nan); // all of it is NaN as soon as a query sees them
        Again which(redo);
        which.seen = rows_of(own_key.odd || own_value.odd);
        for (int i = first; i < end; ++i) {
            const int q0 = lo + (i % tiles) * NQ, hd = kv * a.group + i / tiles;
            const int64_t line0 = ((int64_t)b * a.p.heads + hd) * a.p.queries;
            const auto sees = [&](int query) {
                return key < len && range.holds(query) &&
                       (!a.p.mask || mask_row(a, b, hd, query)[key * a.p.mask_stride[3]] != 0);
            };
            which.look(
                q0, NQ, !a.p.mask && range.covers(q0, NQ),
                [&](int query) {
                    query = min(query, (int)a.p.queries - 1); // as the last tile has it
                    Kinds q, g;
                    q.add(head_row<T>(a.p.q, a.p.q_stride, b, query, hd), dim);
                    g.add(head_row<T>(a.p.dout, a.p.dout_stride, b, query, hd), dim);
                    const float lse = a.row_lse[line0 + query], delta = a.row_delta[line0 + query];
                    return (q.odd || g.odd ? 1u : 0u) | (q.odd || g.odd || lse != lse || not_finite(delta) ? 2u : 0u) |
                           (q.nan || g.all_nan || lse != lse ? 4u : 0u);
                },
                sees);
            for (int x = q0; x < q0 + NQ && (nan_keys & which.rows); ++x)
                which.rows &= ~(nan_keys & rows_of(sees(x)));
        }
        redo = which.which();
    }
    const bool again = (redo >> (lane & 31)) & 1;
    const float scale = (float)a.p.scale;
    const int64_t keys_all = a.p.batch * a.p.kv_heads * a.p.keys;
    const auto part_row = [&](int k) { // [split][dk, dv][batch, kv head, key][DT]
        return a.part + ((int64_t)split * 2 * keys_all + ((int64_t)b * a.p.kv_heads + kv) * a.p.keys + k) * DT;
    };
    if (key < a.p.keys && !again) {
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            if (key >= len) {
                dk[n] = zero16();
                dv[n] = zero16();
            }
            if (a.splits == 1) {
                put_column<T, VEC>(head_row<T>(a.p.dk, a.p.dk_stride, b, key, kv), dk[n], scale, n, h, dim);
                put_column<T, VEC>(head_row<T>(a.p.dv, a.p.dv_stride, b, key, kv), dv[n], kLower, n, h, dim);
            } else {
                put_column<float, true>(part_row(key), dk[n], scale, n, h, DT);
                put_column<float, true>(part_row(key) + keys_all * DT, dv[n], kLower, n, h, DT);
            }
        }
    }
    for (; redo; redo &= redo - 1) {
        const AttnArgs &a = rare_args();
        const int k = key0 + wave * 32 + __builtin_ctzll(redo);
        float ck[2] = {0.0f, 0.0f}, cv[2] = {0.0f, 0.0f};
        for (int i = first; i < end; ++i) {
            const int q0 = lo + (i % tiles) * NQ;
            careful_dkv<T>(a, b, kv * a.group + i / tiles, k, len, q0, min(q0 + NQ, (int)a.p.queries), ck, cv);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int d = lane + 64 * c;
            if (a.splits == 1) {
                if (d < dim) {
                    head_row<T>(a.p.dk, a.p.dk_stride, b, k, kv)[d] = down_apart<T>(ck[c] * scale);
                    head_row<T>(a.p.dv, a.p.dv_stride, b, k, kv)[d] = down_apart<T>(cv[c] * kLower);
                }
            } else if (d < DT) {
                part_row(k)[d] = ck[c] * scale;
                part_row(k)[keys_all * DT + d] = cv[c] * kLower;
            }
        }
    }
}

// ---- dq ------------------------------------------------------------------------
//
// It runs first.  As the forward kernel of many queries: 128 queries of one head in a block, keys and
// values through LDS in tiles of 64 taken as two halves, scores with keys along the rows.
// The sizes of the keys' kernel: 415 to 435 us, 0.94 to 0.99 PFLOP/s of the three products; 17 us.
template <typename T, int DT>
struct QueriesBackward {
    static constexpr int kKeys = 64;
    using TileT = Tile<T, kKeys, DT>;
    static constexpr int kLds = 4 * TileT::kBytes;
};

template <typename T, int DT, bool VEC, Masked MASK>
__global__ __launch_bounds__(256, sizeof(T) == 2 || DT == 32 ? 2 : 1) void attention_queries_backward(AttnArgs a)
{
    using G = QueriesBackward<T, DT>;
    using TileT = typename G::TileT;
    constexpr int KK = DT / 16, ND = DT / 32;
    extern __shared__ __align__(16) uint8_t lds[];

    const uint32_t place = xcd_order(blockIdx.x, a.blocks), block = a.first + place;
    if (place >= a.blocks)
        return;
    const uint32_t q_blocks = (uint32_t)((a.p.queries + 127) / 128);
    const int q0 = (int)(q_blocks - 1 - block % q_blocks) * 128;
    const uint32_t rest = block / q_blocks;
    const int split = (int)(rest % (uint32_t)a.splits);
    const uint32_t bh = rest / (uint32_t)a.splits;
    const int head = (int)(bh % (uint32_t)a.p.heads), b = (int)(bh / (uint32_t)a.p.heads);
    const int kv = head / a.group;

    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6, h = lane >> 5;
    const int query = q0 + wave * 32 + (lane & 31);
    const bool there = query < a.p.queries;
    const int dim = (int)a.p.dim, len = key_length(a, b);
    const Range range = keys_of(a, len, query);
    const uint8_t *mask = nullptr;
    if constexpr (MASK != Masked::none)
        mask = mask_row(a, b, head, min(query, (int)a.p.queries - 1));
    const int64_t line = ((int64_t)b * a.p.heads + head) * a.p.queries + query;

    FragV<T> qf[KK], gf[KK];
    // a row's lse in powers of two (a row that sees nothing: p = 0 everywhere) and D, as the products
    // take them; kept for the keys' kernel, which runs after this one
    float lse = INFINITY, delta = 0.0f;
    {
        const T *q = head_row<T>(a.p.q, a.p.q_stride, b, query, head);
        const T *g = head_row<T>(a.p.dout, a.p.dout_stride, b, query, head);
        const T *o = head_row<T>(static_cast<const void *>(a.p.out), a.p.out_stride, b, query, head);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            qf[kk] = row_from_memory<T, VEC>(q, there, kk, h, dim);
            gf[kk] = row_from_memory<T, VEC>(g, there, kk, h, dim);
            const FragV<T> of = row_from_memory<T, VEC>(o, there, kk, h, dim);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                delta = fmaf(up(gf[kk][e]), up(of[e]), delta);
        }
        delta = pair_sum(delta) * kLower;
        if (there) {
            const float own = a.p.lse[line];
            lse = own == -INFINITY ? INFINITY : own * kLog2e - kLift;
            if (h == 0 && split == 0) {
                a.row_lse[line] = lse;
                a.row_delta[line] = delta;
            }
        }
    }
    float16v dq[ND];
#pragma unroll
    for (int n = 0; n < ND; ++n)
        dq[n] = zero16();
    Lift<T> lift; // of the lane's query; dp and D bring it into ds
    float scaled[2] = {lift.f * kLower, lift.f * delta};

    int lo, hi;
    key_range(a, len, q0, min(q0 + 128, (int)a.p.queries), lo, hi);
    lo &= ~(G::kKeys - 1);
    if (a.splits > 1) {
        const int64_t share = ((hi - lo + a.splits - 1) / a.splits + G::kKeys - 1) / G::kKeys * G::kKeys;
        const int64_t first = least(hi, lo + share * split);
        hi = (int)least(hi, first + share);
        lo = (int)first;
    }
    const T *kbase = head_row<T>(a.p.k, a.p.k_stride, b, 0, kv);
    const T *vbase = head_row<T>(a.p.v, a.p.v_stride, b, 0, kv);
    const int64_t ks = a.p.k_stride[1], vs = a.p.v_stride[1];

    using StageT = Stage<T, G::kKeys, DT, 256, VEC>;
    StageT kst, vst;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        StageT::clear(lds + i * TileT::kBytes, dim, t);
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
    const auto ask = [&](int n, int k) {
        if constexpr (MASK == Masked::ahead)
            words[n].ask(mask, (int)a.p.keys, k + n * 32, h);
    };
    if (lo < hi) {
        fetch(0, len - lo);
        ask(0, lo);
        ask(1, lo);
        store(0);
    }
    loads_done();
    int buf = 0;
    for (int k0 = lo; k0 < hi; k0 += G::kKeys, buf ^= 1) {
        __syncthreads();
        const bool more = k0 + G::kKeys < hi;
        if (more)
            fetch(buf ^ 1, len - k0 - G::kKeys);
        const uint8_t *kl = lds + buf * TileT::kBytes, *vl = lds + (2 + buf) * TileT::kBytes;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int kn = k0 + n * 32;
            if (__all(range.misses(kn, 32))) {
                ask(n, k0 + G::kKeys);
                continue;
            }
            float16v s = zero16(), dp = zero16();
            products_first();
            {
                Pipe<T, 2 * KK, 4> pipe;
                const auto read = [&](int i) {
                    return TileT::row_frag(i < KK ? kl : vl, n * 32 + (lane & 31), i % KK, h);
                };
                pipe.start(read);
                pipe.run(read, [&](int i, const FragV<T> &f) {
                    if (i < KK)
                        s = mma(f, qf[i % KK], s);
                    else
                        dp = mma(f, gf[i % KK], dp);
                });
            }
            settle<T>();
            const auto read = [&](int i) {
                return TileT::col_frag(kl, n * 32 + i / ND * 16, i % ND, lane);
            };
            Pipe<T, 2 * ND, ND == 3 ? 3 : 4> pipe;
            pipe.start(read);
            products_over();
#pragma unroll
            for (int r = 0; r < 16; ++r)
                dp[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale_log2, -lse)) * fmaf(dp[r], scaled[0], -scaled[1]);
            const auto show = [&](int r, bool shown) { dp[r] = shown ? dp[r] : 0.0f; };
            if constexpr (MASK == Masked::ahead) {
                words[n].each_shown((int)a.p.keys, kn, h, show);
                ask(n, k0 + G::kKeys);
            } else if constexpr (MASK == Masked::here) {
                each_shown(mask, a.p.mask_stride[3], (int)a.p.keys, kn, h, show);
            }
            if (!__all(!there || range.covers(kn, 32))) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    dp[r] = range.holds(kn + acc_row(r, h)) ? dp[r] : 0.0f;
            }
            if constexpr (Lift<T>::kOn)
                lift.fit(dp, dq, scaled, 2);
            products_first();
            const FragV<T> ds[2] = {operand<T>(dp, 0), operand<T>(dp, 1)};
            pipe.run(read, [&](int i, const FragV<T> &f) { dq[i % ND] = mma(f, ds[i / ND], dq[i % ND]); });
        }
        if (more)
            store(buf ^ 1);
        if (MASK == Masked::ahead)
            loads_done();
    }

    settle<T>();
    if constexpr (Lift<T>::kOn)
        lift.undo(dq);
    bool bad = false;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            bad |= not_finite(dq[n][i]);
    // D or lse of NaN: so is all of a row that sees a key
    uint64_t redo = rows_of(bad && there && !(lse != lse || (delta != delta && lse < INFINITY)));
    if (redo) {
        const AttnArgs &a = rare_args();
        Again again(redo);
        again.seen = rows_of(not_finite(delta));
        const int64_t step = a.p.mask_stride[3];
        for (int k0 = lo; k0 < hi; k0 += G::kKeys)
            again.look(
                k0, G::kKeys, MASK == Masked::none && range.covers(k0, G::kKeys),
                [&](int key) {
                    key = min(key, len - 1); // as the last tile has it
                    Kinds k, v;
                    k.add(kbase + key * ks, dim);
                    v.add(vbase + key * vs, dim);
                    return (k.odd ? 1u : 0u) | (k.odd || v.odd ? 2u : 0u) | (k.nan || v.nan ? 4u : 0u);
                },
                [&](int key) { return range.holds(key) && (MASK == Masked::none || mask[key * step] != 0); });
        redo = again.which();
    }
    const float scale = (float)a.p.scale;
    const int64_t lines = a.p.batch * a.p.heads * a.p.queries;
    if (there && !((redo >> (lane & 31)) & 1)) {
#pragma unroll
        for (int n = 0; n < ND; ++n) {
            if (a.splits == 1)
                put_column<T, VEC>(head_row<T>(a.p.dq, a.p.dq_stride, b, query, head), dq[n], scale, n, h, dim);
            else
                put_column<float, true>(a.part + (split * lines + line) * DT, dq[n], scale, n, h, DT);
        }
    }
    for (; redo; redo &= redo - 1) {
        const AttnArgs &a = rare_args();
        const int j = __builtin_ctzll(redo), qi = q0 + wave * 32 + j;
        float c[2];
        careful_dq<T>(a, b, head, qi, len, lo, hi, __shfl(lse, j), __shfl(delta, j), c);
        for (int e = 0; e < 2; ++e) {
            const int d = lane + 64 * e;
            if (a.splits == 1) {
                if (d < dim)
                    head_row<T>(a.p.dq, a.p.dq_stride, b, qi, head)[d] = down_apart<T>(c[e] * scale);
            } else if (d < DT) {
                const int64_t ln = ((int64_t)b * a.p.heads + head) * a.p.queries + qi;
                a.part[(split * lines + ln) * DT + d] = c[e] * scale;
            }
        }
    }
}

// The splits' parts summed in their order, of dq, dk and dv in one launch: four columns of a row a
// thread.
struct JoinArgs {
    struct One {
        const float *part;
        void *out;
        int64_t stride[3]; // batch, row, head
        int64_t step;      // from a split's part to the next's
        int64_t lines, rows, heads;
        int splits;
    } one[3];
    int count, dim;
    int64_t first; // the launch's first block of the call's
};

template <typename T, int DT>
__global__ __launch_bounds__(256) void attention_join(JoinArgs j)
{
    const int64_t id = (j.first + blockIdx.x) * 256 + threadIdx.x;
    int64_t line = id / (DT / 4);
    const int d = (int)(id % (DT / 4)) * 4;
    for (int k = 0; k < j.count; ++k) {
        const JoinArgs::One &a = j.one[k];
        if (line >= a.lines) {
            line -= a.lines;
            continue;
        }
        if (d >= j.dim)
            return;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i0 = 0; i0 < a.splits; i0 += 4) {
            float4 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                p[u] = *reinterpret_cast<const float4 *>(a.part + min(i0 + u, a.splits - 1) * a.step + line * DT + d);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u < a.splits)
                    s.x += p[u].x, s.y += p[u].y, s.z += p[u].z, s.w += p[u].w;
        }
        const int64_t bh = line / a.rows;
        T *out = head_row<T>(a.out, a.stride, (int)(bh / a.heads), line - bh * a.rows, (int)(bh % a.heads));
        const float v[4] = {s.x, s.y, s.z, s.w};
        for (int e = 0; e < 4; ++e)
            if (d + e < j.dim)
                out[d + e] = down_apart<T>(v[e]);
        return;
    }
}

template <typename T, int DT, bool VEC>
int run_backward(AttnArgs a, hipStream_t s)
{
    const lic_attention_args &p = a.p;
    float *parts = a.part;
    // two blocks a CU where blocks differ much in length, as in the forward call
    const bool uneven = p.window_left >= 0 || p.window_right >= 0;
    const int q_splits = queries_splits(p), k_splits = keys_splits(p);
    const int64_t q_blocks = (p.queries + 127) / 128 * p.batch * p.heads * q_splits;
    const int64_t k_blocks = (p.keys + 127) / 128 * p.batch * p.kv_heads * k_splits;
    if (q_blocks > kMostBlocks || k_blocks > kMostBlocks)
        return RANS_E_ARG;
    JoinArgs j{};
    j.dim = (int)p.dim;
    const auto joined = [&](const float *part, void *out, const int64_t *stride, int64_t step, int64_t rows,
                            int64_t heads, int splits) {
        j.one[j.count++] = {part, out, {stride[0], stride[1], stride[2]}, step, p.batch * rows * heads, rows, heads,
                            splits};
    };
    if (p.queries > 0) {
        using G = QueriesBackward<T, DT>;
        a.splits = q_splits;
        const int64_t lines = p.batch * p.heads * p.queries;
        a.part = parts;
        const int rc = with_mask<VEC && (sizeof(T) == 4 || DT <= 96)>(p, [&](auto masked) {
            constexpr int kMost = G::kLds > kTwoBlocks ? G::kLds : kTwoBlocks;
            constexpr auto kernel = attention_queries_backward<T, DT, VEC, decltype(masked)::value>;
            if (const int rc = allow_lds<kernel>(kMost))
                return rc;
            in_pieces(q_blocks, 256, [&](int64_t first, uint32_t piece) {
                a.first = (uint32_t)first, a.blocks = piece;
                kernel<<<xcd_grid(piece), 256, uneven ? kMost : G::kLds, s>>>(a);
            });
            return (int)RANS_OK;
        });
        if (rc)
            return rc;
        if (a.splits > 1) {
            joined(parts, p.dq, p.dq_stride, lines * DT, p.queries, p.heads, a.splits);
            parts += a.splits * lines * DT;
        }
    }
    if (p.keys > 0) {
        using G = KeysBackward<T, DT>;
        constexpr int kMost = G::kLds > kTwoBlocks ? G::kLds : kTwoBlocks;
        if (const int rc = allow_lds<attention_keys_backward<T, DT, VEC>>(kMost))
            return rc;
        a.splits = k_splits;
        a.part = parts;
        in_pieces(k_blocks, G::kThreads, [&](int64_t first, uint32_t piece) {
            a.first = (uint32_t)first, a.blocks = piece;
            attention_keys_backward<T, DT, VEC><<<xcd_grid(piece), G::kThreads, uneven ? kMost : G::kLds, s>>>(a);
        });
        if (a.splits > 1) {
            const int64_t all = p.batch * p.kv_heads * p.keys * DT;
            joined(parts, p.dk, p.dk_stride, 2 * all, p.keys, p.kv_heads, a.splits);
            joined(parts + all, p.dv, p.dv_stride, 2 * all, p.keys, p.kv_heads, a.splits);
        }
    }
    if (j.count) {
        int64_t lines = 0;
        for (int k = 0; k < j.count; ++k)
            lines += j.one[k].lines;
        in_pieces((lines * (DT / 4) + 255) / 256, 256, [&](int64_t first, uint32_t piece) {
            j.first = first;
            attention_join<T, DT><<<piece, 256, 0, s>>>(j);
        });
    }
    return launched();
}

}  // namespace
}  // namespace lic
