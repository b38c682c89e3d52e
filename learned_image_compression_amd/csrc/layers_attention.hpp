// layers_attention.hpp -- what the attention kernels share: arguments, the
// tiles in LDS, matrix fragments, and which keys a query sees.
//
// Matrix layout.  All products use 32 x 32 accumulators (64 lanes, 16 values
// each): lane l holds column l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4.  An
// operand fragment is 8 values a lane: row (or column) l % 32 and eight of the
// sixteen summed indexes.  Which eight is free as long as both operands agree:
//
// * "row" fragments (the summed index runs along a tile's row): 8 h .. 8 h + 7
//   of each 16, h = l / 32: one 16-byte read.
// * "column" fragments (it runs down the tile's rows): 4 h .. 4 h + 3 and
//   8 + 4 h .. 8 + 4 h + 3, which is how an accumulator holds its rows.  So the
//   probabilities of one product are the operand of the next as they stand, with
//   no exchange between lanes, and the transposed reads of 4 rows x 16 columns
//   (ds_read_b64_tr_b16) give the other operand.
//
// That is why scores are formed transposed wherever a query's row is reduced: a
// lane then holds one query and half of a tile's keys.
//
// 32-bit tiles use eight 32x32x2 products where 16-bit ones use one 32x32x16.
#pragma once

#include <algorithm>
#include <cmath>

#include "layers_common.hpp"

// m0 is named in a clobber list although the compiler reserves it
#pragma clang diagnostic ignored "-Winline-asm"

namespace lic {

using float16v = float __attribute__((ext_vector_type(16)));
using short4v = short __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    lic_attention_args p;
    float scale_log2;   // scale * log2 e: exponentials are base 2
    float *part;        // split rows: unnormalised sums [split][row][tile dim], then m, l
    float *row_lse;     // backward, [batch][heads][queries] each: lse in powers of two, less 10,
    float *row_delta;   // and dout . out / 2^10
    int splits;
    int group;          // heads that share a kv head
    uint32_t blocks;    // of the launch's real work
    uint32_t first;     // the launch's first block of the call's
};

// The kernel's arguments (its first and only parameter) read again where they are used: what
// only a rare path needs would otherwise be held in scalar registers through the whole
// kernel, and there are too few of them.
__device__ __forceinline__ const AttnArgs &rare_args()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs *)p;
}

template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
    using V = bf16 __attribute__((ext_vector_type(8)));
};
template <>
struct Frag<f16> {
    using V = f16 __attribute__((ext_vector_type(8)));
};
template <>
struct Frag<float> {
    using V = float __attribute__((ext_vector_type(8)));
};
template <typename T>
using FragV = typename Frag<T>::V;

__device__ __forceinline__ float16v mma(FragV<bf16> a, FragV<bf16> b, float16v c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float16v mma(FragV<f16> a, FragV<f16> b, float16v c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float16v mma(FragV<float> a, FragV<float> b, float16v c)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// Waits until the products issued so far are in their registers (at most 18 issue slots
// for 32-bit products, 11 for 16-bit ones).  The hardware leaves that wait to the program and the
// compiler puts it in, but where a branch stands between a product and the first arithmetic on its
// result it may count along the longer path only (seen with hipcc 7.2: 4 slots of 18 on the path
// around an if).  So results are settled before such a branch; arithmetic would wait anyhow.
template <typename T>
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (sizeof(T) == 4)
        asm volatile("s_nop 15\n\ts_nop 2");
    else
        asm volatile("s_nop 11");
    __builtin_amdgcn_sched_barrier(0);
}

// Two waves share a SIMD.  All but their exponentials goes first: then it is the other's
// exponentials that fill the gaps, and neither the matrix unit nor the next tile's loads wait
// for them (8160 x 8160 causal, 16 heads of 128: 300 -> 269 us; 8 heads of 32: 153 -> 125, and
// 147 where the tile's end gave way too).
__device__ __forceinline__ void products_first() { __builtin_amdgcn_s_setprio(1); }
__device__ __forceinline__ void products_over() { __builtin_amdgcn_s_setprio(0); }

// row of an accumulator that a lane's value i is
__device__ __forceinline__ constexpr int acc_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// Eight of an accumulator's values (half 0 or 1 of them) as a column operand.
template <typename T>
__device__ __forceinline__ FragV<T> operand(const float16v &p, int half)
{
    FragV<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = down_apart<T>(p[half * 8 + i]);
    return r;
}

__device__ __forceinline__ float16v zero16()
{
    float16v z;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        z[i] = 0.0f;
    return z;
}

// the larger (sum) of a lane's value and of its partner's 32 lanes away
__device__ __forceinline__ float pair_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A tile of ROWS rows of DT values in LDS: blocks of 32 columns, each ROWS rows of
// 64 (16-bit) or 128 bytes whose 16-byte pieces are permuted by the row, so that
// 16 rows' pieces of a row fragment, and 4 rows x 32 columns of a transposed read,
// fall into all banks once.
template <typename T, int ROWS, int DT>
struct Tile {
    static constexpr int kPiece = 16 / sizeof(T);             // values of a piece
    static constexpr int kPieces = 32 / kPiece;               // pieces of a block's row
    static constexpr int kRowBytes = 32 * sizeof(T);
    static constexpr int kBytes = ROWS * DT * sizeof(T);

    static __device__ __forceinline__ int swizzle(int row)
    {
        return sizeof(T) == 2 ? (row >> 2) & 3 : (row >> 1) & 7;
    }
    static __device__ __forceinline__ int at(int row, int block, int piece)
    {
        return (block * ROWS + row) * kRowBytes + ((piece ^ swizzle(row)) << 4);
    }

    // values 16 kk + 8 h .. + 7 of `row`
    static __device__ __forceinline__ FragV<T> row_frag(const uint8_t *lds, int row, int kk, int h)
    {
        FragV<T> f;
        const int block = kk >> 1;
        if constexpr (sizeof(T) == 2) {
            f = *reinterpret_cast<const FragV<T> *>(lds + at(row, block, (kk & 1) * 2 + h));
        } else {
            using Q = float __attribute__((ext_vector_type(4)));
            const Q a = *reinterpret_cast<const Q *>(lds + at(row, block, (kk & 1) * 4 + 2 * h));
            const Q b = *reinterpret_cast<const Q *>(lds + at(row, block, (kk & 1) * 4 + 2 * h + 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = a[i];
                f[4 + i] = b[i];
            }
        }
        return f;
    }

    // column 32 block + l % 32, rows row0 + {4 h .., 8 + 4 h ..}
    static __device__ __forceinline__ FragV<T> col_frag(const uint8_t *lds, int row0, int block, int lane)
    {
        FragV<T> f;
        const int h = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            // a lane's address: 4 columns of one of the 4 rows; its result: its column's 4 rows
            const int j = lane & 15;
            const int row = row0 + 4 * h + (j >> 2);
            const int piece = ((lane >> 4) & 1) * 2 + ((j & 3) >> 1);
            using Lds = __attribute__((address_space(3))) short4v;
            const auto read = [&](int r) {
                const uint8_t *p = lds + at(r, block, piece) + (j & 1) * 8;
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (Lds *)(__attribute__((address_space(3))) void *)p);
            };
            union {
                short4v s[2];
                FragV<T> f;
            } u;
            u.s[0] = read(row);
            u.s[1] = read(row + 8);
            f = u.f;
        } else {
            const int c = lane & 31;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = row0 + acc_row(i, h);
                f[i] = *reinterpret_cast<const float *>(lds + at(row, block, c >> 2) + (c & 3) * 4);
            }
        }
        return f;
    }
};

// N products whose LDS operands are read a batch of B ahead of the products that take
// them.  Left to itself the compiler reads, waits and multiplies one fragment after another,
// which costs an LDS latency a product; the scheduling barriers hold only memory and matrix
// instructions in their batches.  start() may stand well before run().
template <typename T, int N, int B>
struct Pipe {
    static constexpr int kAhead = B < N ? B : N;
    static_assert(N % kAhead == 0, "whole batches");
    FragV<T> f[2][kAhead];

    template <typename Read>
    __device__ __forceinline__ void start(Read &&read)
    {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            f[0][i] = read(i);
        __builtin_amdgcn_sched_barrier(kLet);
    }
    template <typename Read, typename Use>
    __device__ __forceinline__ void run(Read &&read, Use &&use)
    {
#pragma unroll
        for (int b = 0; b < N / kAhead; ++b) {
            if ((b + 1) * kAhead < N) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    f[(b + 1) & 1][i] = read((b + 1) * kAhead + i);
                __builtin_amdgcn_sched_barrier(kLet);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                use(b * kAhead + i, f[b & 1][i]);
            __builtin_amdgcn_sched_barrier(kLet);
        }
    }
    static constexpr int kLet = 0x6; // vector and scalar arithmetic may pass
};

// Each active lane's N bytes at base + at to LDS, at address `to` + N times its lane.
template <int N>
__device__ __forceinline__ void load_lds(uint32_t to, const void *base, uint32_t at)
{
    if constexpr (N == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(to), "v"(at), "s"(base)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                     :
                     : "s"(to), "v"(at), "s"(base)
                     : "memory", "m0");
}

// All loads of the wave so far are done.  Said with the builtin, so the compiler knows: it would
// wait in each turn of a loop for what was loaded before it.
__device__ __forceinline__ void loads_done()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70); // vmcnt 0
    asm volatile("" ::: "memory");
}

// The same for all but the last N loads.
template <int N>
__device__ __forceinline__ void loads_done_but()
{
    static_assert(N < 64, "what the counter holds");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}

// ROWS rows on their way from memory to a tile, by THREADS threads.
//
// With VEC (sizes, strides and addresses allow 16-byte loads) the memory system writes them to
// LDS by itself: no register is held while they are under way, and store() only waits.  A
// wave's 64 pieces land next to each other, so the permutation is in which piece a lane
// asks for.  The load is written out: for the builtin the compiler waits at the next transposed
// read, which cannot be of the same buffer.  store() waits instead, before the barrier.  Rows past
// the last repeat it (their scores are hidden); pieces past the head's size are never written, and
// clear() made them 0.
// Without VEC values pass through registers one by one, rows and columns past the end as 0.
template <typename T, int ROWS, int DT, int THREADS, bool VEC>
struct Stage {
    using TileT = Tile<T, ROWS, DT>;
    static constexpr int kEach = ROWS * DT / TileT::kPiece / THREADS;
    static_assert(kEach * THREADS * TileT::kPiece == ROWS * DT, "tile and threads");
    uint4 r[VEC ? 1 : kEach];

    // which row, block of columns and piece the i-th 16 bytes of thread t are in LDS
    static __device__ __forceinline__ void place(int i, int t, int &row, int &block, int &piece)
    {
        const int e = i * THREADS + t;
        piece = e % TileT::kPieces;
        const int rest = e / TileT::kPieces;
        row = rest % ROWS;
        block = rest / ROWS;
        if constexpr (VEC)
            piece ^= TileT::swizzle(row);
    }

    static __device__ __forceinline__ void clear(uint8_t *lds, int dim, int t)
    {
        if (VEC && dim < DT) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                int row, block, piece;
                place(i, t, row, block, piece);
                if (block * 32 + piece * TileT::kPiece >= dim)
                    *reinterpret_cast<uint4 *>(lds + TileT::at(row, block, piece)) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }

    // Rows from `base` (the same for the whole block), `rows` of them exist.
    __device__ __forceinline__ void fetch(uint8_t *lds, const T *base, int64_t stride, int rows, int dim, int t)
    {
        if constexpr (VEC) {
            if (dim == DT)
                ask<true>(lds, base, stride, rows, dim, t);
            else
                ask<false>(lds, base, stride, rows, dim, t);
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                int row, block, piece;
                place(i, t, row, block, piece);
                const int d = block * 32 + piece * TileT::kPiece;
                const T *p = base + (int64_t)row * stride + d;
                Vec<T, TileT::kPiece> v;
#pragma unroll
                for (int e = 0; e < TileT::kPiece; ++e)
                    v.v[e] = row < rows && d + e < dim ? p[e] : (T)0.0f;
                r[i] = *reinterpret_cast<const uint4 *>(&v);
            }
        }
    }

    template <bool WHOLE>
    static __device__ __forceinline__ void ask(uint8_t *lds, const T *base, int64_t stride, int rows, int dim, int t)
    {
        // the wave's first piece; lane l's lands 16 l bytes on
        const uint32_t first = __builtin_amdgcn_readfirstlane(
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + (t & ~63) * 16);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            int row, block, piece;
            place(i, t, row, block, piece);
            const int d = block * 32 + piece * TileT::kPiece;
            const uint32_t at = (uint32_t)min(row, rows - 1) * (uint32_t)(stride * sizeof(T)) + d * sizeof(T);
            if (WHOLE || d < dim)
                load_lds<16>(first + i * THREADS * 16, base, at);
        }
    }

    // what fetch() asked for is in LDS (after this and a barrier)
    __device__ __forceinline__ void store(uint8_t *lds, int t) const
    {
        if constexpr (VEC) {
            loads_done();
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                int row, block, piece;
                place(i, t, row, block, piece);
                *reinterpret_cast<uint4 *>(lds + TileT::at(row, block, piece)) = r[i];
            }
        }
    }
};

// One row's values 16 kk + 8 h .. + 7 straight from memory (0 beyond dim or without a row).
template <typename T, bool VEC>
__device__ __forceinline__ FragV<T> row_from_memory(const T *row, bool there, int kk, int h, int dim)
{
    FragV<T> f;
    const int d = 16 * kk + 8 * h;
    if constexpr (VEC) {
        constexpr int P = 16 / sizeof(T);
        using Q = T __attribute__((ext_vector_type(P)));
#pragma unroll
        for (int i = 0; i < 8; i += P) {
            Q q;
#pragma unroll
            for (int e = 0; e < P; ++e)
                q[e] = (T)0.0f;
            if (there && d + i < dim)
                q = *reinterpret_cast<const Q *>(row + d + i);
#pragma unroll
            for (int e = 0; e < P; ++e)
                f[i + e] = q[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = there && d + i < dim ? row[d + i] : (T)0.0f;
    }
    return f;
}

// The keys that one query may see by lengths and windows, or the queries that may see
// one key: [first, first + count).
struct Range {
    int first;
    uint32_t count;

    __device__ __forceinline__ void set(int64_t lo, int64_t hi, int64_t end)
    {
        first = (int)least(lo, end);
        count = hi > lo ? (uint32_t)(hi - lo) : 0u;
    }
    __device__ __forceinline__ bool holds(int x) const { return (uint32_t)(x - first) < count; }
    // whether all (none) of [x0, x0 + n) are in it
    __device__ __forceinline__ bool covers(int x0, int n) const
    {
        return x0 >= first && (int64_t)x0 + n <= (int64_t)first + count;
    }
    __device__ __forceinline__ bool misses(int x0, int n) const
    {
        return count == 0u || (int64_t)x0 + n <= first || x0 >= (int64_t)first + count;
    }
};

// Keys that any of the queries [q0, q1) may see: [lo, hi).
__device__ __forceinline__ void key_range(const AttnArgs &a, int len, int q0, int q1, int &lo, int &hi)
{
    const int64_t t0 = (int64_t)q0 + len - a.p.queries, t1 = (int64_t)q1 - 1 + len - a.p.queries;
    const int64_t l = a.p.window_left < 0 ? 0 : most(0, t0 - a.p.window_left);
    const int64_t h = a.p.window_right < 0 ? len : least(len, t1 + a.p.window_right + 1);
    lo = (int)least(l, len);
    hi = (int)most(h, lo);
}

// Queries that may see any of the keys [k0, k1): [lo, hi).
__device__ __forceinline__ void query_range(const AttnArgs &a, int len, int k0, int k1, int &lo, int &hi)
{
    const int64_t back = (int64_t)len - a.p.queries; // position - query
    const int64_t l = a.p.window_right < 0 ? 0 : most(0, (int64_t)k0 - a.p.window_right - back);
    const int64_t h = a.p.window_left < 0 ? a.p.queries : least(a.p.queries, (int64_t)k1 + a.p.window_left - back);
    lo = (int)least(l, a.p.queries);
    hi = (int)most(h, lo);
}

__device__ __forceinline__ Range keys_of(const AttnArgs &a, int len, int query)
{
    Range r;
    int lo, hi;
    key_range(a, len, query, query + 1, lo, hi);
    r.set(lo, query < a.p.queries ? hi : lo, len);
    return r;
}

__device__ __forceinline__ Range queries_of(const AttnArgs &a, int len, int key)
{
    Range r;
    int lo, hi;
    query_range(a, len, key, key + 1, lo, hi);
    r.set(lo, key < len ? hi : lo, a.p.queries);
    return r;
}

__device__ __forceinline__ int key_length(const AttnArgs &a, int b)
{
    const int keys = (int)a.p.keys;
    return a.p.key_lengths ? min(max(a.p.key_lengths[b], 0), keys) : keys;
}

__device__ __forceinline__ const uint8_t *mask_row(const AttnArgs &a, int b, int head, int query)
{
    return a.p.mask + b * a.p.mask_stride[0] + head * a.p.mask_stride[1] +
           (int64_t)query * a.p.mask_stride[2];
}

// The mask's entries of an accumulator's 16 pairs, at x0 + its row of `extent` >= 4 in all, where they
// lie next to each other.  Of each 32 a lane reads one half at once and gives its partner 32 lanes away the
// words that are the partner's: reading its own four words costs four times as many accesses to
// scattered lines.  The last entries are read word by word; one past the extent, which the range
// hides, reads one before it instead.
struct MaskWords {
    uint32_t word[4];

    __device__ __forceinline__ void ask(const uint8_t *mask, int extent, int x0, int h)
    {
        if (x0 + 32 <= extent) {
            __builtin_memcpy(word, mask + x0 + 16 * h, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_memcpy(&word[i], mask + min(x0 + 4 * h + 8 * i, extent - 4), 4);
        }
    }
    // f(i, whether the mask shows it); the words are spent
    template <typename F>
    __device__ __forceinline__ void each_shown(int extent, int x0, int h, F &&f)
    {
        if (x0 + 32 <= extent) {
            // words 0 .. 3 of the lower lane, 4 .. 7 of the upper: 0 2 4 6 and 1 3 5 7
            const auto a = __builtin_amdgcn_permlane32_swap(word[0], word[1], false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(word[2], word[3], false, false);
            word[0] = a[0], word[1] = b[0], word[2] = a[1], word[3] = b[1];
        } else { // a word at the end began before its pairs: what it has of them comes down
#pragma unroll
            for (int i = 0; i < 4; ++i)
                word[i] >>= 8 * min(max(x0 + 4 * h + 8 * i - (extent - 4), 0), 3);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f(i, (word[i >> 2] & (0xffu << (8 * (i & 3)))) != 0u);
    }
};
__host__ __device__ __forceinline__ bool mask_in_words(int64_t step, int64_t extent)
{
    return step == 1 && extent >= 4;
}

// How the kernels that hold queries take a mask: there is none; in words, asked for a tile ahead; where
// they need it.  Each has its own instance, since registers bound them.  (Forward, us, here / ahead,
// float16: 4 x 8 heads of 32, 1000 x 1000 32 / 27; 8 x 8 of 64, 2048 x 2048 176 / 155; 2 x 8 of 96, 2040 x 2040 83 / 67;
// 2 x 3 of 64, 4080 x 4080 68 / 80, since only two blocks fit a CU; without a mask 8 x 8 of 64 take 93.)
enum class Masked { none, ahead, here };

// f(i, whether the mask shows it) for an accumulator's 16 pairs, at x0 + its row of `extent` in
// all.  mask: the entry of 0, `step` bytes to the next.  All entries are asked for before the first
// is looked at.  (32 x 6 heads of 256 x 256, forward: 37 us with single bytes.)
template <typename F>
__device__ __forceinline__ void each_shown(const uint8_t *mask, int64_t step, int extent, int x0, int h, F &&f)
{
    if (mask_in_words(step, extent)) {
        MaskWords words;
        words.ask(mask, extent, x0, h);
        words.each_shown(extent, x0, h, f);
        return;
    }
    const int x = x0 + 4 * h;
    uint8_t byte[16];
    if (x0 + 32 <= extent) {
        const uint8_t *p = mask + x * step;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            byte[i] = p[acc_row(i, 0) * step];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            byte[i] = mask[min(x + acc_row(i, 0), extent - 1) * step];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        f(i, byte[i] != 0);
}

template <typename T>
__device__ __forceinline__ const T *head_row(const void *p, const int64_t *stride, int b, int64_t row, int head)
{
    return static_cast<const T *>(p) + b * stride[0] + row * stride[1] + head * stride[2];
}
template <typename T>
__device__ __forceinline__ T *head_row(void *p, const int64_t *stride, int b, int64_t row, int head)
{
    return static_cast<T *>(p) + b * stride[0] + row * stride[1] + head * stride[2];
}

// Blocks are handed to the 8 XCDs in turn; neighbours in this order share an XCD and
// so its L2, which lets the blocks of one head read its keys from there.
__device__ __forceinline__ uint32_t xcd_order(uint32_t block, uint32_t blocks)
{
    const uint32_t each = (blocks + 7) / 8;
    return (block & 7) * each + (block >> 3); // may be >= blocks: no work
}
inline uint32_t xcd_grid(uint32_t blocks) { return (blocks + 7) / 8 * 8; }
// blocks of a call that its kernels count
constexpr int64_t kMostBlocks = 0x7fffff00;

// Orders a wave's own LDS writes before its other lanes' reads.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) <= 3.402823466e38f); }

// The rows (a lane's l % 32) where either of a row's two lanes says so.
__device__ __forceinline__ uint64_t rows_of(bool flag)
{
    const uint64_t f = __builtin_amdgcn_ballot_w64(flag);
    return (f | (f >> 32)) & 0xffffffffull;
}

// Whether a row holds a NaN, only NaN, or anything that is not finite.
struct Kinds {
    bool nan = false, all_nan = true, odd = false;

    template <typename T>
    __device__ __forceinline__ void add(const T *row, int dim)
    {
        for (int d = 0; d < dim; ++d) {
            const float x = up(row[d]);
            nan |= x != x, all_nan &= x != x, odd |= not_finite(x);
        }
    }
};

// Which of a wave's results that are not finite (rows: a lane's l % 32) have to be formed again.  Hidden
// pairs have p = 0, but 0 times a NaN or an infinity of theirs is NaN.  So a row is right as it is if it
// sees something that makes all of its values NaN whatever is hidden, or if it sees something that
// is not finite and nothing hidden is.  The others, and those that see only finite numbers (sums too
// large in 32 bits), are formed again, at hundreds of times the cost.
struct Again {
    static constexpr unsigned kStains = 1, kOdd = 2, kAllNan = 4; // where it is hidden; where it is seen
    uint64_t rows, seen = 0, hidden = 0;

    __device__ __forceinline__ explicit Again(uint64_t bad) : rows(bad) {}

    // What the rows do or do not see at [x, x + n), n <= 64: kind(x) of what is there, sees(x) whether the
    // lane's row does.  all: the lane's row sees all of it.
    template <typename Kind, typename Sees>
    __device__ __forceinline__ void look(int x, int n, bool all, Kind &&kind, Sees &&sees)
    {
        const int lane = threadIdx.x & 63;
        const bool mine = (rows >> (lane & 31)) & 1;
        if (!(rows & ~seen) && __all(all || !mine))
            return;
        const unsigned k = lane < n ? kind(x + lane) : 0u;
        const uint64_t stains = __builtin_amdgcn_ballot_w64((k & kStains) != 0);
        const uint64_t all_nan = __builtin_amdgcn_ballot_w64((k & kAllNan) != 0);
        for (uint64_t at = __builtin_amdgcn_ballot_w64(k != 0); at && rows; at &= at - 1) {
            const int j = __builtin_ctzll(at);
            const uint64_t they = rows_of(sees(x + j));
            seen |= they;
            if ((stains >> j) & 1)
                hidden |= ~they;
            if ((all_nan >> j) & 1)
                rows &= ~they;
        }
    }
    __device__ __forceinline__ uint64_t which() const { return rows & (hidden | ~seen); }
};

// A lane's part of an accumulator's column, times f, to columns 32 block .. of a row.
template <typename T, bool VEC>
__device__ __forceinline__ void put_column(T *out, const float16v &v, float f, int block, int h, int dim)
{
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const int d = block * 32 + acc_row(i, h);
        Vec<T, 4> w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w.v[e] = down_apart<T>(v[i + e] * f);
        if constexpr (VEC) {
            if (d < dim)
                *reinterpret_cast<Vec<T, 4> *>(out + d) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < dim)
                    out[d + e] = w.v[e];
        }
    }
}

// Per element type; defined in one translation unit each (layers_attention_<type>.hip).
template <typename T>
struct Attention {
    static int forward(AttnArgs a, hipStream_t s);
    static int backward(AttnArgs a, hipStream_t s);
};

constexpr int kTwoBlocks = 64 * 1024; // of LDS: two blocks fit a CU's 160 KiB, three do not

// ROOM: whether the 8 registers that words ahead take are there without spills.
template <bool ROOM, typename F>
int with_mask(const lic_attention_args &p, F &&f)
{
    using std::integral_constant;
    if (!p.mask)
        return f(integral_constant<Masked, Masked::none>{});
    if constexpr (ROOM) {
        if (mask_in_words(p.mask_stride[3], p.keys))
            return f(integral_constant<Masked, Masked::ahead>{});
    }
    return f(integral_constant<Masked, Masked::here>{});
}

// Splits of the key axis that the rows kernel takes: two blocks a CU, at least 256 keys
// each, at most 64.
inline int row_splits(const lic_attention_args &p)
{
    const int64_t rows = p.queries * (p.heads / p.kv_heads);
    const int64_t blocks = (rows + 31) / 32 * p.batch * p.kv_heads;
    int64_t n = 512 / blocks;
    const int64_t most = (p.keys + 255) / 256;
    n = n < most ? n : most;
    n = n < 64 ? n : 64;
    return n < 1 ? 1 : (int)n;
}

// Which forward kernel: the one of few queries (32 rows of all heads that share keys a block) or the
// one of many (128 queries of one head a block), and into how many splits of the key axis.  The
// estimate, in us, fitted to measured calls of 1 to 1024 blocks: the first gets through 1000 tiles of
// 32 x 32 in `row`; a CU of the second takes `unit` for a block's 64 keys, `pair` times that for two
// blocks'; parts of a join are written and read from the caches at 8 TB/s.  It is within 12% of the
// best choice for nearly all of 165 calls and sizes measured, and splits are taken where they gain 7%.
// Measured (us, few / many / many with splits), bfloat16, dim 64: 8160 x 8160, 1 head 41 / 127 / 38 of 8;
// 1000 x 1000, 8 heads 15 / 20 / 16 of 4; 510 x 510, 24 heads 10 / 13 / 16 of 2; 8160 x 8160, 6 heads
// - / 169 / 143 of 4; the same causal, 4 heads - / 122 / 65 of 4; 2048 x 2048, 64 heads - / 93 / 113 of 2.
struct ForwardPlan {
    bool few;
    int splits;
};

inline ForwardPlan forward_plan(const lic_attention_args &p)
{
    const double nd = (double)((p.dim + 31) / 32), queries = (double)p.queries, keys = (double)p.keys;
    const bool f32 = p.dtype == LIC_F32, left = p.window_left >= 0, right = p.window_right >= 0;
    const double row = f32 ? 0.15 + 1.3 * nd : 0.3 + 0.044 * nd * nd;
    const double unit = f32 ? 0.4 + 2.1 * nd : 0.65 + 0.15 * nd;
    const double pair = f32 ? 1.95 : 1.1 + 0.17 * nd;
    // keys that a row sees at most, and the part of them that a row sees on average
    const double most = left && right ? std::min(keys, (double)(p.window_left + p.window_right) + 128.0) : keys;
    const double part = left == right ? 1.0 : queries < keys ? 1.0 - 0.5 * queries / keys : 0.5 * keys / queries;

    const int64_t row_tiles = (p.queries * (p.heads / p.kv_heads) + 31) / 32 * p.batch * p.kv_heads;
    const int row_split = row_splits(p);
    const double turns = std::min(1.0, (double)(row_tiles * row_split) / 512.0); // wide heads: a block a CU
    const double few = (double)row_tiles * most / 32000.0 * row * (part < 1.0 ? 0.85 : 1.0) + 5.3 +
                       (f32 ? 2.0 : 0.55) * nd * nd * turns + (row_split > 1 ? 4.0 : 0.0);

    const int64_t blocks = (p.queries + 127) / 128 * p.batch * p.heads, tiles = (int64_t)most / 64 + 1;
    int best = 1;
    double many = 0.0;
    for (int n = 1; n <= 16 && (n == 1 || (blocks * n <= 2048 && tiles >= 4 * n)); n *= 2) {
        const double share = (double)((tiles + n - 1) / n) * unit;
        const double each = (double)(blocks * n) / 256.0; // blocks of a CU
        const int64_t whole = (blocks * n + 255) / 256;
        const double even = (double)(whole / 2) * pair + (double)(whole % 2);
        const double uneven = std::max(each > 1.0 ? 0.5 + 0.5 * pair : 1.0, each * part * pair / 2.0);
        const double join = n == 1 ? 0.0 : 6.0 + 1e-6 * n * (double)(p.batch * p.heads) * queries * 32.0 * nd;
        const double cost = (4.0 + share * (part < 1.0 ? uneven : even) + join) * (n == 1 ? 0.93 : 1.0);
        if (n == 1 || cost < many)
            best = n, many = cost;
    }
    return few < many ? ForwardPlan{true, row_split} : ForwardPlan{false, best};
}

// Splits of the backward kernels' loops (over the query tiles of all heads that share a kv head, and over
// key tiles), by the same kind of estimate: blocks, a block's steps, the time of a step, `at_once` blocks
// on a CU, the floats of one split's parts.  Causal order makes blocks of very different length,
// which more of them even out (8160 x 8160 causal, 16 heads of 128 on 4: dk, dv 612 us with 512 blocks,
// 892 with 256); a split costs its part's way through memory.
// Measured (both kernels and join, us, with 1 / 2 / 4 / 8 splits of keys' blocks): float, 4 x 6 heads of 32,
// 510 x 510 70 / 54 / 55 / 58; bfloat16, 8 heads of 64, 1000 x 1000 50 / 42 / 39 / 42; 8 x 8 heads of 64, 510 x 510
// causal 36 / 46 / 55 / 76; 4 heads of 64, 4080 x 4080 149 / 107 / 93 / 105.
inline int backward_splits(const lic_attention_args &p, int at_once, int64_t blocks, double steps, double unit,
                           double floats)
{
    const double nd = (double)((p.dim + 31) / 32);
    const double pair = at_once == 1 ? 2.0 : p.dtype == LIC_F32 ? 1.95 : 1.1 + 0.17 * nd;
    const bool one_sided = (p.window_left >= 0) != (p.window_right >= 0);
    const double queries = (double)p.queries, keys = (double)p.keys;
    const double part = !one_sided ? 1.0 : queries < keys ? 1.0 - 0.5 * queries / keys : 0.5 * keys / queries;
    int best = 1;
    double least = 0.0;
    for (int n = 1; n <= 16 && (n == 1 || (double)(2 * n) <= steps); n += part < 1.0 ? n : 1) {
        const double each = (double)(blocks * n) / 256.0;
        const int64_t whole = (blocks * n + 255) / 256;
        const double even = (double)(whole / 2) * pair + (double)(whole % 2);
        const double uneven = std::max(each > 1.0 && at_once > 1 ? 0.5 + 0.5 * pair : 1.0, each * part * pair / 2.0);
        const double load = part < 1.0 ? uneven : even;
        const double join = n == 1 ? 0.0 : 4.0 + 1e-6 * n * floats;
        const double cost = (load * (1.5 + std::ceil(steps / n) * unit) + join) * (n == 1 ? 0.93 : 1.0);
        if (n == 1 || cost < least)
            best = n, least = cost;
    }
    return best;
}
// rows of `all` that one of the other kind sees at most
inline double rows_seen(const lic_attention_args &p, int64_t all)
{
    const bool both = p.window_left >= 0 && p.window_right >= 0;
    return both ? std::min((double)all, (double)(p.window_left + p.window_right) + 128.0) : (double)all;
}
inline int keys_splits(const lic_attention_args &p)
{
    const double nd = (double)((p.dim + 31) / 32), group = (double)(p.heads / p.kv_heads);
    const bool f32 = p.dtype == LIC_F32;
    return backward_splits(p, p.dim <= (f32 ? 32 : 96) ? 2 : 1, (p.keys + 127) / 128 * p.batch * p.kv_heads,
                           std::ceil(rows_seen(p, p.queries) / 32.0) * group, f32 ? 2.3 * nd : 0.7 + 0.07 * nd,
                           64.0 * nd * (double)(p.batch * p.kv_heads * p.keys));
}
inline int queries_splits(const lic_attention_args &p)
{
    const double nd = (double)((p.dim + 31) / 32);
    const bool f32 = p.dtype == LIC_F32;
    return backward_splits(p, !f32 || p.dim <= 32 ? 2 : 1, (p.queries + 127) / 128 * p.batch * p.heads,
                           std::ceil(rows_seen(p, p.keys) / 64.0), f32 ? 4.0 * nd : 1.2 + 0.2 * nd,
                           32.0 * nd * (double)(p.batch * p.heads * p.queries));
}

}  // namespace lic
