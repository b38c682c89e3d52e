// layers_linear.hip -- linear attention's C entry points (checks, workspace, jobs), the step of single
// tokens, and the sums over heads that share keys.
#include "layers_linear.hpp"

namespace lic {
namespace {

// ---- single tokens --------------------------------------------------------------
//
// S' = g S + k v',  out = scale q S'.  The state's way through memory bounds it: a block takes a head's
// state, a thread four of its columns (one where value_dim does not divide) of every R-th row; out is added
// up over the R threads of a column in LDS, in their order.  A long memory's g is 1 + expm1f(log g) in two parts: its
// rounding to 32 bits would be the same at every step, up to 3e-5 of the state after a thousand of them.  16 x 16 heads of
// 64 on 4, bfloat16: 6.1 us (8.4 MB of states).
constexpr int kStepThreads = 256;

struct StepArgs {
    lic_linear_attention_args p;
    int32_t share, across, down; // heads of a kv head; threads of a state's row; rows at once
    uint32_t first;
};

template <typename T, int V>
__global__ __launch_bounds__(kStepThreads) void linear_step(StepArgs a)
{
    __shared__ float sums[kStepThreads * V];
    const lic_linear_attention_args &p = a.p;
    const uint32_t line = a.first + blockIdx.x;
    const int b = (int)(line / (uint32_t)p.heads), head = (int)(line - (uint32_t)b * (uint32_t)p.heads), kv = head / a.share;
    const int t = (int)threadIdx.x, row0 = t / a.across, e = (t - row0 * a.across) * V;
    const bool live = !p.lengths || p.lengths[b] > 0;
    const T *q = head_row<T>(p.q, p.q_stride, b, 0, head), *k = head_row<T>(p.k, p.k_stride, b, 0, kv);
    const T *v = head_row<T>(p.v, p.v_stride, b, 0, kv);
    const float *state = p.state ? p.state + b * p.state_stride[0] + head * p.state_stride[1] + e : nullptr;
    float *last = p.state_out ? p.state_out + b * p.state_out_stride[0] + head * p.state_out_stride[1] + e : nullptr;
    const float log_decay = p.log_decay[head], scale = (float)p.scale, more = expm1f(log_decay);
    const bool near_one = fabsf(log_decay) < 0.5f;
    const float g = near_one ? 1.0f + more : expf(log_decay), rest = near_one ? more - (g - 1.0f) : 0.0f;
    using VT = Vec<float, V>;
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        o[i] = 0.0f;
    if (row0 < a.down) {
        float ve[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            ve[i] = live ? up(v[e + i]) : 0.0f;
        constexpr int U = 4; // rows asked for at once
        for (int d0 = row0; d0 < p.dim; d0 += U * a.down) {
            VT s[U];
            float qd[U], kd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int d = d0 + u * a.down;
                s[u] = VT{};
                qd[u] = kd[u] = 0.0f;
                if (d < p.dim) {
                    if (state)
                        s[u] = load_at<VT>(state + d * p.state_stride[2]);
                    if (live) {
                        qd[u] = up(q[d]);
                        kd[u] = up(k[d]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int d = d0 + u * a.down;
                if (d >= p.dim)
                    break;
                if (live) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float before = s[u].v[i], low = not_finite(before) ? 0.0f : before * rest;
                        s[u].v[i] = fmaf(before, g, fmaf(kd[u], ve[i], low));
                        o[i] = fmaf(qd[u], s[u].v[i], o[i]);
                    }
                }
                if (last)
                    store_at(last + d * p.state_out_stride[2], s[u]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            sums[row0 * (a.across * V) + e + i] = o[i];
    }
    __syncthreads();
    if (t < p.value_dim) {
        float s = 0.0f;
        for (int r = 0; r < a.down; ++r)
            s += sums[r * (a.across * V) + t];
        head_row<T>(p.out, p.out_stride, b, 0, head)[t] = down_apart<T>(live ? s * scale : 0.0f);
    }
}

template <typename T, int V>
int run_step(StepArgs a, hipStream_t s)
{
    a.across = (int)((a.p.value_dim + V - 1) / V);
    a.down = std::min<int>(kStepThreads / a.across, (int)a.p.dim);
    in_pieces(a.p.batch * a.p.heads, kStepThreads, [&](int64_t first, uint32_t blocks) {
        a.first = (uint32_t)first;
        linear_step<T, V><<<blocks, kStepThreads, 0, s>>>(a);
    });
    return launched();
}

// ---- sums over heads that share ---------------------------------------------------

// dk and dv in one launch: their parts [batch][kv head][share][token][dim], four values a thread where they divide.
// Memory bounds it: four heads of 128 to each of 4, 8160 tokens, 25 us (6.0 TB/s of 150 MB).
struct JoinArgs {
    const float *part[2];
    void *out[2];
    int64_t out_stride[2][3];
    int64_t total[2]; // threads of each
    int32_t dim[2];
    int64_t tokens, first;
    int32_t heads, share;
};

template <typename T, int V>
__global__ __launch_bounds__(256) void linear_join(JoinArgs a)
{
    using VT = Vec<float, V>;
    int64_t id = (a.first + blockIdx.x) * 256 + threadIdx.x;
    const int which = id >= a.total[0];
    if (which)
        id -= a.total[0];
    if (id >= a.total[which])
        return;
    const int dim = a.dim[which], units = dim / V;
    const int64_t row = id / units, line = row / a.tokens; // (batch, kv head)
    const int d = (int)(id - row * units) * V;
    const int64_t token = row - line * a.tokens, step = a.tokens * dim;
    const float *part = a.part[which] + line * a.share * step + token * dim + d;
    VT s = load_at<VT>(part);
    for (int i = 1; i < a.share; ++i) {
        const VT o = load_at<VT>(part + i * step);
#pragma unroll
        for (int e = 0; e < V; ++e)
            s.v[e] += o.v[e];
    }
    const int64_t b = line / a.heads;
    Vec<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e)
        o.v[e] = down<T>(s.v[e]);
    store_at(head_row<T>(a.out[which], a.out_stride[which], (int)b, token, (int)(line - b * a.heads)) + d, o);
}

// dlog_decay[head]: one wave a head, over the batch's parts (its segments).
__global__ __launch_bounds__(64) void linear_decay_join(const double *sums, float *out, int32_t batch, int32_t heads, int32_t parts)
{
    const int head = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int64_t i = lane; i < (int64_t)batch * parts; i += 64) {
        const int64_t b = i / parts;
        s += sums[(b * heads + head) * parts + (i - b * parts)];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        s += __shfl_xor(s, d);
    if (lane == 0)
        out[head] = (float)s;
}

// ---- the states before the segments ------------------------------------------------
//
// start_(k+1) = g^(tokens of k) start_k + what k adds, in place of what the segments add.  A block takes all
// segments of 1024 / GROUPS numbers of a state, four a thread, in GROUPS groups of up to EACH neighbours.  Each
// group adds up its own, then what comes from the groups before it, so a thread waits for memory once.  (The
// powers are formed in 64 bits, by one wave of the block: by all of them they were most of its time.  Rounded to 32
// bits they would be off the same way at every segment: by 5e-6 of the state behind 255 segments of 128 tokens.)
// Memory bounds it: 16 states of 128 x 128 for each of 16 heads 10 us (33 MB read and written); 32 of 64 x 64 for 32, 10.
constexpr int kMostSegments = 256;

struct ScanArgs {
    LinearJob job[2];
    const float *log_decay;
    const int32_t *lengths;
    int64_t tokens, first;
    int32_t heads, jobs, segments, each, start_floats, tiles; // a block's share of a state
    int32_t blocks;                                           // of 32 columns
    int32_t group;                                            // segments of a group
};

// g^n in two parts of 32 bits, the second above 0 where the first is, so an infinity times both is one.
struct Power {
    float whole, rest;
    static __device__ __forceinline__ Power of(float log_decay, int n)
    {
        const double p = n == 0 ? 1.0 : exp((double)log_decay * n);
        float whole = (float)p;
        if (!(whole > 0.0f) || not_finite(whole)) // 0, NaN, infinity
            return {whole, whole};
        whole = (double)whole < p ? whole : __uint_as_float(__float_as_uint(whole) - 1);
        return {whole, (float)(p - (double)whole)};
    }
    static __device__ __forceinline__ Power one() { return {1.0f - 0x1p-24f, 0x1p-24f}; }
    // v g^n + add
    __device__ __forceinline__ float times(float v, float add) const { return fmaf(v, whole, fmaf(v, rest, add)); }
};

template <int EACH, int GROUPS>
__global__ __launch_bounds__(256) void linear_scan(ScanArgs a)
{
    constexpr int ACROSS = 256 / GROUPS;
    using VT = Vec<float, 4>;
    __shared__ VT ends[GROUPS][ACROSS];
    __shared__ Power powers[2 + GROUPS]; // of a whole segment, of the last one in use, of each group
    const int64_t id = a.first + blockIdx.x, line = id / a.tiles / a.jobs;
    const int tile = (int)(id % a.tiles), which = (int)(id / a.tiles % a.jobs);
    const LinearJob &p = a.job[which];
    const int b = (int)(line / a.heads), head = (int)(line - (int64_t)b * a.heads);
    const int t = (int)threadIdx.x, x = t % ACROSS, group = t / ACROSS;
    const int at = (tile * ACROSS + x) * 4; // its numbers of a state: four rows of a column of StateImage
    const int place = at / 4 / 64, lane = at / 4 & 63, fours = place / a.blocks;
    const int row0 = 32 * (fours >> 2) + state_row(8 * (fours & 3) + 4 * (lane >> 5));
    const int column = 32 * (place % a.blocks) + (lane & 31);
    float *starts = p.starts + line * a.segments * a.start_floats + at;
    // in the order of time: segment 0 first, or the last one
    const auto index = [&](int k) { return p.reverse ? a.segments - 1 - k : k; };
    const int k0 = group * a.group, adding = a.segments - (p.last ? 0 : 1);
    VT add[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        add[i] = VT{};
        if (i < a.group && k0 + i < adding)
            add[i] = load_at<VT>(starts + (int64_t)index(k0 + i) * a.start_floats);
    }
    VT run{};
    if (group == 0 && p.first && column < p.dim_z) {
        const float *first = p.first + b * p.first_stride[0] + head * p.first_stride[1] + column * p.first_stride[3];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < p.dim_x)
                run.v[i] = first[(row0 + i) * p.first_stride[2]];
    }
    const int all = a.lengths ? min(max(a.lengths[b], 0), (int)a.tokens) : (int)a.tokens;
    const auto tokens_of = [&](int k) { return min(max(all - index(k) * a.each, 0), a.each); };
    if (t < 64) {
        int n = t == 0 ? a.each : all % a.each;
        if (t >= 2) { // a group's, in time
            const int from = min((t - 2) * a.group, a.segments), to = min(from + a.group, a.segments);
            n = min(max(all - (p.reverse ? a.segments - to : from) * a.each, 0), (to - from) * a.each);
        }
        const Power power = Power::of(a.log_decay[head], n);
        if (t < 2 + GROUPS)
            powers[t] = power;
    }
    __syncthreads();
    const Power whole = powers[0], part = powers[1];
    const auto power = [&](int k) {
        const int n = tokens_of(k);
        return n == a.each ? whole : n == 0 ? Power::one() : part;
    };
    VT sum = run;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (i < a.group && k0 + i < a.segments) {
            const Power g = power(k0 + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum.v[e] = g.times(sum.v[e], add[i].v[e]);
        }
    ends[group][x] = sum;
    __syncthreads();
    if (group > 0) {
        run = ends[0][x];
        for (int k = 1; k < group; ++k) {
            const Power g = powers[2 + k];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                run.v[e] = g.times(run.v[e], ends[k][x].v[e]);
        }
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (i < a.group && k0 + i < a.segments) {
            store_at(starts + (int64_t)index(k0 + i) * a.start_floats, run);
            const Power g = power(k0 + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                run.v[e] = g.times(run.v[e], add[i].v[e]);
        }
    if (p.last && k0 < a.segments && k0 + a.group >= a.segments && column < p.dim_z) { // behind the last one
        float *last = p.last + b * p.last_stride[0] + head * p.last_stride[1] + column * p.last_stride[3];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < p.dim_x)
                last[(row0 + i) * p.last_stride[2]] = run.v[i];
    }
}

int run_scan(const LinearArgs &l, hipStream_t s)
{
    ScanArgs a{};
    for (int i = 0; i < l.jobs; ++i)
        a.job[i] = l.job[i];
    a.log_decay = l.log_decay, a.lengths = l.lengths, a.tokens = l.tokens;
    a.heads = l.heads, a.jobs = l.jobs, a.segments = l.segments, a.each = l.each, a.start_floats = l.start_floats;
    a.blocks = (std::max(l.job[0].dim_x, l.job[0].dim_z) + 31) / 32;
    const auto run = [&](auto kernel, int each, int groups) {
        a.group = std::min(each, (l.segments + groups - 1) / groups);
        a.tiles = l.start_floats / (1024 / groups);
        in_pieces((int64_t)l.batch * l.heads * l.jobs * a.tiles, 256, [&](int64_t first, uint32_t blocks) {
            a.first = first;
            kernel<<<blocks, 256, 0, s>>>(a);
        });
    };
    if (l.segments <= 4)
        run(linear_scan<4, 1>, 4, 1);
    else if (l.segments <= 16)
        run(linear_scan<4, 4>, 4, 4);
    else if (l.segments <= 64)
        run(linear_scan<4, 16>, 4, 16);
    else
        run(linear_scan<16, 16>, 16, 16);
    return launched();
}

// ---- entries -------------------------------------------------------------------------

bool valid(const lic_linear_attention_args *p)
{
    const auto in = [](int64_t v, int64_t least, int64_t most) { return v >= least && v <= most; };
    return p && valid_dtype(p->dtype) && in(p->batch, 0, 1 << 20) && in(p->tokens, 0, 1 << 28) &&
           in(p->kv_heads, 1, 65536) && in(p->heads, p->kv_heads, 65536) && p->heads % p->kv_heads == 0 &&
           in(p->dim, 1, LIC_MAX_HEAD_DIM) && in(p->value_dim, 1, LIC_MAX_HEAD_DIM) &&
           p->batch * p->heads <= (1ll << 28) && p->batch * p->heads * p->tokens <= (1ll << 33);
}

bool ok(const int64_t *s) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }

bool valid_call(const lic_linear_attention_args &p, bool backward)
{
    if (!ok(p.q_stride) || !ok(p.k_stride) || !ok(p.v_stride) || !(p.scale > 0.0) || !(p.scale < 1e30) || !p.log_decay ||
        (p.state && !ok(p.state_stride)))
        return false;
    if (p.tokens > 0 && (!p.q || !p.k || !p.v))
        return false;
    if (!backward)
        return ok(p.out_stride) && (p.tokens == 0 || p.out) && (!p.state_out || ok(p.state_out_stride));
    return ok(p.dout_stride) && ok(p.dq_stride) && ok(p.dk_stride) && ok(p.dv_stride) &&
           (p.tokens == 0 || (p.dout && p.dq && p.dk && p.dv)) && (!p.dstate || ok(p.dstate_stride)) &&
           (!p.dstate_in || ok(p.dstate_in_stride));
}

uint64_t round256(uint64_t n) { return (n + 255) / 256 * 256; }

// How the tokens are split: into as many segments as make four blocks a CU, each of at least 64 tokens.  A state's way
// through scratch memory (written, scanned, read) is as long as that of 4 * dim tokens' rows, so heads wider than
// 64 take one block a CU.  Measured (us, with 256 / 512 / 1024 / 1536 blocks): forward, bfloat16, 2 x 16 heads of 64, 8160
// tokens 117 / 81 / 62 / 75; 6 heads of 32, 32640 tokens 81 / 52 / 41 / 42; trained, 16 heads of 128, 8160 tokens 409 / 439 /
// 532 / 607; float, 4 x 6 heads of 32, 510 tokens in segments of 510 / 128 / 64 / 32: 200 / 120 / 64 / 68.
struct Split {
    int32_t segments, each;
    explicit Split(const lic_linear_attention_args &p)
    {
        const int64_t want = std::max(p.dim, p.value_dim) <= 64 ? 1024 : 256;
        int64_t n = want / std::max<int64_t>(p.batch * p.heads, 1);
        n = std::max<int64_t>(1, std::min<int64_t>(n, kMostSegments));
        each = (int32_t)std::max<int64_t>(2 * kRun, ((p.tokens + n - 1) / n + kRun - 1) / kRun * kRun);
        segments = (int32_t)std::max<int64_t>(1, (p.tokens + each - 1) / each);
    }
};

int32_t start_floats(const lic_linear_attention_args &p)
{
    const int32_t wide = (int32_t)(std::max(p.dim, p.value_dim) + 31) / 32 * 32;
    return wide * wide;
}

// Scratch memory of a call: the states before segments (and their gradients behind them), parts of dk and
// dv, sums of dlog_decay.
struct Layout {
    uint64_t starts, ends, dk, dv, sums, bytes;
    Layout(const lic_linear_attention_args &p, bool backward)
    {
        const Split split(p);
        const uint64_t lines = (uint64_t)p.batch * p.heads, shared = backward && p.heads > p.kv_heads;
        const uint64_t states = split.segments > 1 ? round256(lines * split.segments * start_floats(p) * 4) : 0;
        starts = 0;
        ends = starts + states;
        dk = ends + (backward ? states : 0);
        dv = dk + (shared ? round256(lines * p.tokens * p.dim * 4) : 0);
        sums = dv + (shared ? round256(lines * p.tokens * p.value_dim * 4) : 0);
        bytes = sums + (backward ? round256(lines * split.segments * 8) : 0);
    }
};

// Whether rows may be fetched 16 bytes at a time.  One tensor that may not be sends all of a call through loads of a value,
// at about three times the time (bfloat16, 2 x 16 heads of 64, 8160 tokens: 58 us, 190 with v 2 bytes off, 241 with
// value_dim 65).
template <typename T>
bool vector_rows(const lic_linear_attention_args &p, const void *x, const int64_t *stride, int64_t heads)
{
    constexpr int n = 16 / sizeof(T);
    return !x || (aligned_to(x, 16) && (p.batch == 1 || stride[0] % n == 0) && (p.tokens == 1 || stride[1] % n == 0) &&
                  stride[1] < (1 << 24) && (heads == 1 || stride[2] % n == 0));
}

void set3(int64_t *to, const int64_t *from) { std::copy(from, from + 3, to); }
// a state's strides with its rows and columns in their order, or the other way round
void set_state(int64_t *to, const int64_t *from, bool turned)
{
    to[0] = from[0], to[1] = from[1];
    to[2] = turned ? 1 : from[2], to[3] = turned ? from[2] : 1;
}

LinearArgs common(const lic_linear_attention_args &p)
{
    const Split split(p);
    LinearArgs a{};
    a.segments = split.segments;
    a.each = split.each;
    a.start_floats = start_floats(p);
    a.log_decay = p.log_decay;
    a.lengths = p.lengths;
    a.tokens = p.tokens;
    a.batch = (int32_t)p.batch;
    a.heads = (int32_t)p.heads;
    a.scale = (float)p.scale;
    return a;
}

// The states before the segments of the first `jobs` jobs.
template <typename T>
int make_states(LinearArgs a, int jobs, bool vec, hipStream_t s)
{
    a.jobs = jobs;
    if (const int rc = Linear<T>::states(a, vec, s))
        return rc;
    return run_scan(a, s);
}

template <typename T>
int forward(const lic_linear_attention_args &p, void *ws, hipStream_t s)
{
    const int32_t share = (int32_t)(p.heads / p.kv_heads);
    if (p.tokens == 1) {
        StepArgs a{};
        a.p = p;
        a.share = share;
        return p.value_dim % 4 == 0 ? run_step<T, 4>(a, s) : run_step<T, 1>(a, s);
    }
    constexpr int n = 16 / sizeof(T);
    const bool vec = p.dim % n == 0 && p.value_dim % n == 0 && vector_rows<T>(p, p.q, p.q_stride, p.heads) &&
                     vector_rows<T>(p, p.k, p.k_stride, p.kv_heads) && vector_rows<T>(p, p.v, p.v_stride, p.kv_heads) &&
                     vector_rows<T>(p, p.out, p.out_stride, p.heads);
    LinearArgs a = common(p);
    LinearJob &j = a.job[0];
    a.jobs = 1;
    j.x = p.q, j.y = p.k, j.z = p.v, j.out = p.out, j.first = p.state, j.last = p.state_out;
    set3(j.x_stride, p.q_stride), set3(j.y_stride, p.k_stride), set3(j.z_stride, p.v_stride);
    set3(j.out_stride, p.out_stride);
    set_state(j.first_stride, p.state_stride, false), set_state(j.last_stride, p.state_out_stride, false);
    j.x_share = 1, j.y_share = j.z_share = share;
    j.dim_x = (int32_t)p.dim, j.dim_z = (int32_t)p.value_dim;
    j.read = a.scale, j.write = 1.0f;
    j.starts = static_cast<float *>(ws);
    if (a.segments > 1) {
        if (const int rc = make_states<T>(a, 1, vec, s))
            return rc;
        j.last = nullptr;
    }
    return Linear<T>::sweep(a, vec, s);
}

template <typename T>
int join(const lic_linear_attention_args &p, const float *dk, const float *dv, hipStream_t s)
{
    JoinArgs a{};
    a.part[0] = dk, a.part[1] = dv;
    a.out[0] = p.dk, a.out[1] = p.dv;
    set3(a.out_stride[0], p.dk_stride), set3(a.out_stride[1], p.dv_stride);
    a.dim[0] = (int32_t)p.dim, a.dim[1] = (int32_t)p.value_dim;
    a.tokens = p.tokens;
    a.heads = (int32_t)p.kv_heads;
    a.share = (int32_t)(p.heads / p.kv_heads);
    const int vec = p.dim % 4 == 0 && p.value_dim % 4 == 0 ? 4 : 1;
    for (int i = 0; i < 2; ++i)
        a.total[i] = p.batch * p.kv_heads * p.tokens * (a.dim[i] / vec);
    in_pieces((a.total[0] + a.total[1] + 255) / 256, 256, [&](int64_t first, uint32_t blocks) {
        a.first = first;
        if (vec == 4)
            linear_join<T, 4><<<blocks, 256, 0, s>>>(a);
        else
            linear_join<T, 1><<<blocks, 256, 0, s>>>(a);
    });
    return launched();
}

template <typename T>
int backward(const lic_linear_attention_args &p, void *ws, hipStream_t s)
{
    constexpr int n = 16 / sizeof(T);
    const bool vec = p.dim % n == 0 && p.value_dim % n == 0 && vector_rows<T>(p, p.q, p.q_stride, p.heads) &&
                     vector_rows<T>(p, p.k, p.k_stride, p.kv_heads) && vector_rows<T>(p, p.v, p.v_stride, p.kv_heads) &&
                     vector_rows<T>(p, p.dout, p.dout_stride, p.heads) && vector_rows<T>(p, p.dq, p.dq_stride, p.heads) &&
                     vector_rows<T>(p, p.dk, p.dk_stride, p.kv_heads) && vector_rows<T>(p, p.dv, p.dv_stride, p.kv_heads);
    const Layout at(p, true);
    uint8_t *base = static_cast<uint8_t *>(ws);
    const int32_t share = (int32_t)(p.heads / p.kv_heads);
    LinearArgs a = common(p);
    a.jobs = 3;
    const auto job = [&](int i, const void *x, const int64_t *xs, int32_t x_share, const void *y, const int64_t *ys,
                         int32_t y_share, const void *z, const int64_t *zs, int32_t z_share, void *out,
                         const int64_t *os, int64_t dim_x, int64_t dim_z) -> LinearJob & {
        LinearJob &j = a.job[i];
        j.x = x, j.y = y, j.z = z, j.out = out;
        set3(j.x_stride, xs), set3(j.y_stride, ys), set3(j.z_stride, zs), set3(j.out_stride, os);
        j.x_share = x_share, j.y_share = y_share, j.z_share = z_share;
        j.dim_x = (int32_t)dim_x, j.dim_z = (int32_t)dim_z;
        j.reverse = i > 0;
        j.read = i > 0 ? 1.0f : a.scale, j.write = i > 0 ? a.scale : 1.0f;
        j.first = i > 0 ? p.dstate : p.state;
        j.starts = reinterpret_cast<float *>(base + (i > 0 ? at.ends : at.starts));
        return j;
    };
    LinearJob &dq = job(0, p.dout, p.dout_stride, 1, p.v, p.v_stride, share, p.k, p.k_stride, share, p.dq, p.dq_stride,
                        p.value_dim, p.dim);
    set_state(dq.first_stride, p.state_stride, true);
    dq.turned = 1;
    LinearJob &dv = job(1, p.k, p.k_stride, share, p.q, p.q_stride, 1, p.dout, p.dout_stride, 1, p.dv, p.dv_stride, p.dim,
                        p.value_dim);
    set_state(dv.first_stride, p.dstate_stride, false);
    dv.last = p.dstate_in;
    set_state(dv.last_stride, p.dstate_in_stride, false);
    LinearJob &dk = job(2, p.v, p.v_stride, share, p.dout, p.dout_stride, 1, p.q, p.q_stride, 1, p.dk, p.dk_stride,
                        p.value_dim, p.dim);
    set_state(dk.first_stride, p.dstate_stride, true);
    dk.turned = 1;
    if (a.segments > 1) {
        LinearArgs st = a; // the states themselves, as the forward call's, and their gradients, as dv's
        LinearJob &j = st.job[0];
        j.y = p.k, j.z = p.v;
        set3(j.y_stride, p.k_stride), set3(j.z_stride, p.v_stride);
        set_state(j.first_stride, p.state_stride, false);
        j.dim_x = (int32_t)p.dim, j.dim_z = (int32_t)p.value_dim;
        if (const int rc = make_states<T>(st, 2, vec, s))
            return rc;
        dv.last = nullptr;
    }
    if (share > 1) {
        dk.part = reinterpret_cast<float *>(base + at.dk);
        dv.part = reinterpret_cast<float *>(base + at.dv);
    }
    if (const int rc = Linear<T>::sweep(a, vec, s))
        return rc;
    if (share > 1 && p.tokens > 0) {
        if (const int rc = join<T>(p, dk.part, dv.part, s))
            return rc;
    }
    if (!p.dlog_decay)
        return RANS_OK;
    DecayArgs d{};
    d.q = p.q, d.k = p.k, d.v = p.v, d.dout = p.dout, d.state = p.state, d.dstate = p.dstate;
    d.sums = reinterpret_cast<double *>(base + at.sums);
    d.starts = reinterpret_cast<float *>(base + at.starts);
    d.ends = reinterpret_cast<float *>(base + at.ends);
    d.segments = a.segments, d.each = a.each, d.start_floats = a.start_floats;
    set3(d.q_stride, p.q_stride), set3(d.k_stride, p.k_stride), set3(d.v_stride, p.v_stride);
    set3(d.dout_stride, p.dout_stride), set3(d.state_stride, p.state_stride), set3(d.dstate_stride, p.dstate_stride);
    d.log_decay = p.log_decay, d.lengths = p.lengths, d.tokens = p.tokens;
    d.batch = (int32_t)p.batch, d.heads = (int32_t)p.heads, d.share = share;
    d.dim = (int32_t)p.dim, d.value_dim = (int32_t)p.value_dim, d.scale = a.scale;
    if (const int rc = Linear<T>::decay(d, vec, s))
        return rc;
    linear_decay_join<<<(uint32_t)p.heads, 64, 0, s>>>(d.sums, p.dlog_decay, d.batch, d.heads, d.segments);
    return launched();
}

int call(const lic_linear_attention_args *args, void *ws, uint64_t ws_bytes, hipStream_t s, bool back)
{
    if (!valid(args))
        return RANS_E_ARG;
    const lic_linear_attention_args &p = *args;
    if (p.batch == 0 && !(back && p.dlog_decay))
        return RANS_OK;
    if (p.batch == 0) { // a sum over nothing
        linear_decay_join<<<(uint32_t)p.heads, 64, 0, s>>>(nullptr, p.dlog_decay, 0, (int32_t)p.heads, 1);
        return launched();
    }
    if (!valid_call(p, back))
        return RANS_E_ARG;
    const uint64_t need = Layout(p, back).bytes;
    if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need))
        return RANS_E_WORKSPACE;
    return with_dtype(p.dtype, [&](auto t) {
        using T = decltype(t);
        return back ? backward<T>(p, ws, s) : forward<T>(p, ws, s);
    });
}

}  // namespace
}  // namespace lic

extern "C" uint64_t lic_linear_attention_workspace_bytes(const lic_linear_attention_args *args, int32_t backward)
{
    return lic::valid(args) ? lic::Layout(*args, backward != 0).bytes : 0;
}

extern "C" int lic_linear_attention_forward(const lic_linear_attention_args *args, void *workspace,
                                            uint64_t workspace_bytes, hipStream_t hstream)
{
    return lic::call(args, workspace, workspace_bytes, hstream, false);
}

extern "C" int lic_linear_attention_backward(const lic_linear_attention_args *args, void *workspace,
                                             uint64_t workspace_bytes, hipStream_t hstream)
{
    return lic::call(args, workspace, workspace_bytes, hstream, true);
}
