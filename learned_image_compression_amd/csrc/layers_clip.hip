// layers_clip.hip -- the global norm of many tensors' values, and their scaling by it.
//
//   norm = sqrt(sum of x^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c x
//
// HBM bounds it: every value is read twice, the second time from the last-level cache where
// they fit, and written once.  Two launches a list of 120 tensors (their addresses are kernel
// arguments, so nothing is copied to the device and a captured graph holds them): sums of a block's
// chunks in 64 bits; then every block adds all sums up itself, in one order, which is cheaper
// than a launch in between, and scales its chunks, the last ones first, since they are what
// the caches still hold.  With c = 1 and out = x there is nothing left to do.
//
// Measured: 138M bfloat16 values in 56 tensors 51 us for the sums (5.4 TB/s), 90 us to scale them (6.1 TB/s read
// and written); 410000 float values in 16 tensors 4.3 and 4.9 us, which are launches.
#include <algorithm>
#include <utility>
#include <vector>

#include "layers_common.hpp"

namespace lic {
namespace {

constexpr int kClipThreads = 256;
constexpr int kTensors = 120;                 // of a launch
constexpr int64_t kChunkBytes = 16 * 1024;    // four vectors a thread
constexpr int kSums = 1024;                   // blocks of a call's sums: four a CU

struct ClipList {
    const void *x[kTensors];
    void *out[kTensors];
    int64_t n_type[kTensors];        // values, and their type in the lowest two bits
    uint32_t first[kTensors + 1];    // chunks before each tensor's
    uint32_t blocks;
    int32_t count;
};
struct ClipArgs {
    double *sums;    // of the launch
    const double *all;
    float *norm;
    double max_norm;
    uint32_t all_sums;
    bool past, write_norm;
};
static_assert(sizeof(ClipList) + sizeof(ClipArgs) <= 4096, "kernel arguments");

int64_t chunk_values(int64_t dtype) { return kChunkBytes / dtype_bytes(dtype); }

// the chunks of this block, f(tensor, its values' type, first value, end)
template <bool DOWN, typename F>
__device__ __forceinline__ void each_chunk(const ClipList &l, F &&f)
{
    const uint32_t chunks = l.first[l.count];
    const uint32_t lo = (uint32_t)((uint64_t)chunks * blockIdx.x / gridDim.x);
    const uint32_t hi = (uint32_t)((uint64_t)chunks * (blockIdx.x + 1) / gridDim.x);
    int t = 0;
    for (uint32_t i = lo; i < hi; ++i) {
        const uint32_t k = DOWN ? lo + hi - 1 - i : i;
        if (i == lo || k < l.first[t] || k >= l.first[t + 1]) { // the last tensor that begins at or before k
            int a = 0, z = l.count;
            while (z - a > 1) {
                const int m = (a + z) / 2;
                if (l.first[m] <= k)
                    a = m;
                else
                    z = m;
            }
            t = a;
        }
        const int64_t n = l.n_type[t] >> 2;
        const int type = (int)(l.n_type[t] & 3);
        const int64_t each = kChunkBytes / (type == LIC_F32 ? 4 : 2), at = (int64_t)(k - l.first[t]) * each;
        f(t, type, at, at + each < n ? at + each : n);
    }
}

template <typename T>
__device__ __forceinline__ double squares(const T *x, int64_t n)
{
    constexpr int V = 16 / sizeof(T), EACH = (int)(kChunkBytes / 16 / kClipThreads);
    using VT = Vec<T, V>;
    double s = 0.0;
    const int t = (int)threadIdx.x;
    if (n == kChunkBytes / (int64_t)sizeof(T)) {
        VT v[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            v[e] = load_at<VT>(x + (e * kClipThreads + t) * V);
#pragma unroll
        for (int e = 0; e < EACH; ++e)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const double d = (double)up(v[e].v[i]);
                s = fma(d, d, s);
            }
        return s;
    }
    const int whole = (int)(n / V);
    for (int u = t; u < whole; u += kClipThreads) {
        const VT v = load_at<VT>(x + u * V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double d = (double)up(v.v[i]);
            s = fma(d, d, s);
        }
    }
    if (t < (int)n - whole * V) {
        const double d = (double)up(x[whole * V + t]);
        s = fma(d, d, s);
    }
    return s;
}

template <typename T>
__device__ __forceinline__ void scaled(const T *x, T *out, int64_t n, float before, float c, bool past)
{
    constexpr int V = 16 / sizeof(T), EACH = (int)(kChunkBytes / 16 / kClipThreads);
    using VT = Vec<T, V>;
    const auto times = [&](VT v) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v.v[i] = down_apart<T>(up(v.v[i]) * before * c);
        return v;
    };
    const int t = (int)threadIdx.x;
    if (n == kChunkBytes / (int64_t)sizeof(T)) {
        VT v[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            v[e] = load_at<VT>(x + (e * kClipThreads + t) * V);
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            store_at(out + (e * kClipThreads + t) * V, times(v[e]), past);
        return;
    }
    const int whole = (int)(n / V);
    for (int u = t; u < whole; u += kClipThreads)
        store_at(out + u * V, times(load_at<VT>(x + u * V)), past);
    if (t < (int)n - whole * V)
        out[whole * V + t] = down_apart<T>(up(x[whole * V + t]) * before * c);
}

// the sum over the block, the same for all of its threads
__device__ __forceinline__ double block_total(double s)
{
    __shared__ double waves[kClipThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0)
        waves[threadIdx.x >> 6] = s;
    __syncthreads();
    s = waves[0];
#pragma unroll
    for (int w = 1; w < kClipThreads / 64; ++w)
        s += waves[w];
    return s;
}

__global__ __launch_bounds__(kClipThreads) void clip_sums(ClipList l, ClipArgs a)
{
    double s = 0.0;
    each_chunk<false>(l, [&](int t, int type, int64_t at, int64_t end) {
        switch (type) {
        case LIC_F32: s += squares(static_cast<const float *>(l.x[t]) + at, end - at); break;
        case LIC_F16: s += squares(static_cast<const f16 *>(l.x[t]) + at, end - at); break;
        default: s += squares(static_cast<const bf16 *>(l.x[t]) + at, end - at); break;
        }
    });
    s = block_total(s);
    if (threadIdx.x == 0)
        a.sums[blockIdx.x] = s;
}

__device__ __forceinline__ double total_norm(const ClipArgs &a)
{
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < a.all_sums; i += kClipThreads)
        s += a.all[i];
    const double norm = sqrt(block_total(s));
    if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0)
        *a.norm = (float)norm;
    return norm;
}

__global__ __launch_bounds__(kClipThreads) void clip_norm(ClipArgs a) { total_norm(a); }

__global__ __launch_bounds__(kClipThreads) void clip_scale(ClipList l, ClipArgs a)
{
    const double part = a.max_norm / (total_norm(a) + 1e-6);
    // a factor that 32 bits hold in a few bits or not at all takes its power of two first
    const float before = part < 0x1p-64 ? 0x1p-64f : 1.0f;
    const float c = part >= 1.0 ? 1.0f : (float)(part / (double)before); // NaN stays
    each_chunk<true>(l, [&](int t, int type, int64_t at, int64_t end) {
        if (c == 1.0f && l.x[t] == l.out[t])
            return;
        switch (type) {
        case LIC_F32:
            scaled(static_cast<const float *>(l.x[t]) + at, static_cast<float *>(l.out[t]) + at, end - at, before, c,
                   a.past);
            break;
        case LIC_F16:
            scaled(static_cast<const f16 *>(l.x[t]) + at, static_cast<f16 *>(l.out[t]) + at, end - at, before, c, a.past);
            break;
        default:
            scaled(static_cast<const bf16 *>(l.x[t]) + at, static_cast<bf16 *>(l.out[t]) + at, end - at, before, c, a.past);
            break;
        }
    });
}

bool valid(const lic_gradient *g, int64_t count)
{
    if (count < 0 || count > (1 << 24) || (count > 0 && !g))
        return false;
    for (int64_t i = 0; i < count; ++i)
        if (!valid_dtype(g[i].dtype) || g[i].n < 0 || g[i].n > (1ll << 40) || (g[i].n > 0 && !g[i].x))
            return false;
    return true;
}

// Whether an output overlaps another or an input that is not its own.
bool apart(const lic_gradient *g, int64_t count)
{
    struct Part {
        uint64_t from, to;
        int64_t owner;
        bool out;
    };
    std::vector<Part> parts;
    parts.reserve(2 * (size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        const uint64_t bytes = (uint64_t)g[i].n * dtype_bytes(g[i].dtype);
        if (bytes == 0)
            continue;
        const uint64_t x = (uint64_t)(uintptr_t)g[i].x, out = (uint64_t)(uintptr_t)g[i].out;
        if (x != out) {
            parts.push_back({x, x + bytes, i, false});
            if (x < out + bytes && out < x + bytes)
                return false;
        }
        parts.push_back({out, out + bytes, i, true});
    }
    std::sort(parts.begin(), parts.end(), [](const Part &a, const Part &b) { return a.from < b.from; });
    uint64_t any = 0, outs = 0; // ends of what came before
    for (const Part &p : parts) {
        if (p.from < outs || (p.out && p.from < any))
            return false;
        any = std::max(any, p.to);
        if (p.out)
            outs = std::max(outs, p.to);
    }
    return true;
}

struct Plan {
    std::vector<ClipList> lists;
    uint32_t sums = 0;
    uint64_t bytes = 0;
};

// Lists of tensors with values, at most 2^31 chunks each; a tensor of more is several.
Plan plan_of(const lic_gradient *g, int64_t count)
{
    Plan plan;
    ClipList l{};
    const auto flush = [&] {
        if (l.count)
            plan.lists.push_back(l);
        l = ClipList{};
    };
    constexpr int64_t most = 1ll << 30; // chunks of an entry, and of a list before its last entry
    for (int64_t i = 0; i < count; ++i) {
        const int64_t each = chunk_values(g[i].dtype), size = dtype_bytes(g[i].dtype);
        plan.bytes += (uint64_t)(g[i].n * size);
        for (int64_t at = 0; at < g[i].n; at += most * each) {
            const int64_t n = std::min(g[i].n - at, most * each);
            if (l.count == kTensors || l.first[l.count] >= (uint32_t)most)
                flush();
            l.x[l.count] = static_cast<const uint8_t *>(g[i].x) + at * size;
            l.out[l.count] = g[i].out ? static_cast<uint8_t *>(g[i].out) + at * size : nullptr;
            l.n_type[l.count] = n << 2 | g[i].dtype;
            l.first[l.count + 1] = l.first[l.count] + (uint32_t)((n + each - 1) / each);
            ++l.count;
        }
    }
    flush();
    const uint32_t each = std::max<uint32_t>(128, kSums / std::max<uint32_t>(1, (uint32_t)plan.lists.size()));
    for (ClipList &list : plan.lists) {
        list.blocks = std::min(list.first[list.count], each);
        plan.sums += list.blocks;
    }
    return plan;
}

int call(const lic_gradient *g, int64_t count, double max_norm, float *norm, void *ws, uint64_t ws_bytes,
         hipStream_t s, bool scale)
{
    if (!valid(g, count) || !norm || !(max_norm >= 0.0) || !(max_norm < 1e300))
        return RANS_E_ARG;
    if (scale) {
        for (int64_t i = 0; i < count; ++i)
            if (g[i].n > 0 && !g[i].out)
                return RANS_E_ARG;
        if (!apart(g, count))
            return RANS_E_ARG;
    }
    const Plan plan = plan_of(g, count);
    if (plan.sums > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < plan.sums * sizeof(double)))
        return RANS_E_WORKSPACE;
    ClipArgs a{};
    a.all = static_cast<const double *>(ws);
    a.norm = norm;
    a.max_norm = max_norm;
    a.all_sums = plan.sums;
    a.past = 2 * plan.bytes > (uint64_t)kCacheBytes;
    a.sums = static_cast<double *>(ws);
    for (const ClipList &l : plan.lists) {
        clip_sums<<<l.blocks, kClipThreads, 0, s>>>(l, a);
        a.sums += l.blocks;
    }
    a.write_norm = true;
    if (!scale || plan.lists.empty()) {
        clip_norm<<<1, kClipThreads, 0, s>>>(a);
        return launched();
    }
    for (auto l = plan.lists.rbegin(); l != plan.lists.rend(); ++l) {
        const uint32_t blocks = std::min<uint32_t>(l->first[l->count], 2 * kSums);
        clip_scale<<<blocks, kClipThreads, 0, s>>>(*l, a);
        a.write_norm = false;
    }
    return launched();
}

// C++ exceptions (of memory that is not there) end at the C entries.
template <typename F>
int guarded(F &&f)
{
    try {
        return f();
    } catch (...) {
        return RANS_E_HIP;
    }
}

}  // namespace
}  // namespace lic

extern "C" uint64_t lic_clip_gradients_workspace_bytes(const lic_gradient *tensors, int64_t count)
{
    if (!lic::valid(tensors, count))
        return 0;
    try {
        return lic::plan_of(tensors, count).sums * sizeof(double);
    } catch (...) {
        return 0;
    }
}

extern "C" int lic_gradient_norm(const lic_gradient *tensors, int64_t count, float *norm, void *workspace,
                                 uint64_t workspace_bytes, hipStream_t hstream)
{
    return lic::guarded(
        [&] { return lic::call(tensors, count, 0.0, norm, workspace, workspace_bytes, hstream, false); });
}

extern "C" int lic_clip_gradients(const lic_gradient *tensors, int64_t count, double max_norm, float *norm,
                                  void *workspace, uint64_t workspace_bytes, hipStream_t hstream)
{
    return lic::guarded(
        [&] { return lic::call(tensors, count, max_norm, norm, workspace, workspace_bytes, hstream, true); });
}
