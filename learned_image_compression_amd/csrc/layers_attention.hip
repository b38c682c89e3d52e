// layers_attention.hip -- attention's C entry points: checks, workspace, element type.
#include "layers_attention.hpp"

namespace lic {
namespace {

// Extents that every index of the kernels (32 bits for rows and pairs' blocks) holds.
bool valid(const lic_attention_args *p)
{
    const auto in = [](int64_t v, int64_t least, int64_t most) { return v >= least && v <= most; };
    return p && valid_dtype(p->dtype) && in(p->batch, 0, 1 << 20) && in(p->queries, 0, 1 << 28) &&
           in(p->keys, 0, 1 << 28) && in(p->kv_heads, 1, 65536) && in(p->heads, p->kv_heads, 65536) &&
           p->heads % p->kv_heads == 0 && in(p->dim, 1, LIC_MAX_HEAD_DIM) &&
           p->queries * (p->heads / p->kv_heads) <= (1ll << 30) && in(p->window_left, -1, 1ll << 40) &&
           in(p->window_right, -1, 1ll << 40) &&
           p->batch * p->heads * p->queries <= (1ll << 33) && p->batch * p->kv_heads * p->keys <= (1ll << 33);
}

bool valid_call(const lic_attention_args &p, bool backward)
{
    const auto ok = [](const int64_t *s) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; };
    if (!ok(p.q_stride) || !ok(p.k_stride) || !ok(p.v_stride) || !ok(p.out_stride) ||
        (p.mask && (!ok(p.mask_stride) || p.mask_stride[3] < 0)) || !(p.scale > 0.0) || !(p.scale < 1e30))
        return false;
    if (p.queries > 0 && (!p.q || !p.out || !p.lse))
        return false;
    if (p.keys > 0 && (!p.k || !p.v))
        return false;
    if (!backward)
        return true;
    return ok(p.dout_stride) && ok(p.dq_stride) && ok(p.dk_stride) && ok(p.dv_stride) &&
           (p.queries == 0 || (p.dout && p.dq)) && (p.keys == 0 || (p.dk && p.dv));
}

uint64_t round256(uint64_t n) { return (n + 255) / 256 * 256; }

uint64_t row_bytes(const lic_attention_args &p)
{
    return round256((uint64_t)p.batch * p.heads * p.queries * 2 * sizeof(float));
}

// Parts of split sums are as wide as the widest tile the call may take.
uint64_t part_bytes(const lic_attention_args &p, bool backward)
{
    const uint64_t q_lines = (uint64_t)p.batch * p.heads * p.queries;
    const uint64_t k_lines = (uint64_t)p.batch * p.kv_heads * p.keys;
    if (!backward) {
        const int n = forward_plan(p).splits;
        return n > 1 ? n * q_lines * (LIC_MAX_HEAD_DIM + 2) * 4 : 0;
    }
    const int nk = keys_splits(p), nq = queries_splits(p);
    return (nk > 1 ? 2 * nk * k_lines * LIC_MAX_HEAD_DIM * 4 : 0) + (nq > 1 ? nq * q_lines * LIC_MAX_HEAD_DIM * 4 : 0);
}

uint64_t workspace(const lic_attention_args &p, bool backward)
{
    if (p.batch == 0 || (p.queries == 0 && !backward))
        return 0;
    return (backward ? row_bytes(p) : 0) + round256(part_bytes(p, backward));
}

int call(const lic_attention_args *args, void *ws, uint64_t ws_bytes, hipStream_t s, bool backward)
{
    if (!valid(args) || args->batch == 0)
        return args && args->batch == 0 && valid(args) ? RANS_OK : RANS_E_ARG;
    if (!valid_call(*args, backward))
        return RANS_E_ARG;
    if (args->queries == 0 && (!backward || args->keys == 0))
        return RANS_OK;
    const uint64_t need = workspace(*args, backward);
    if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need))
        return RANS_E_WORKSPACE;
    AttnArgs a{};
    a.p = *args;
    a.scale_log2 = (float)(args->scale * 1.4426950408889634);
    a.group = (int)(args->heads / args->kv_heads);
    a.splits = 1;
    if (backward) {
        a.row_lse = static_cast<float *>(ws);
        a.row_delta = a.row_lse + args->batch * args->heads * args->queries;
        a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + row_bytes(*args));
    } else {
        a.part = static_cast<float *>(ws);
    }
    return with_dtype(args->dtype, [&](auto t) {
        using T = decltype(t);
        return backward ? Attention<T>::backward(a, s) : Attention<T>::forward(a, s);
    });
}

}  // namespace
}  // namespace lic

extern "C" uint64_t lic_attention_workspace_bytes(const lic_attention_args *args, int32_t backward)
{
    return lic::valid(args) ? lic::workspace(*args, backward != 0) : 0;
}

extern "C" int lic_attention_forward(const lic_attention_args *args, void *workspace, uint64_t workspace_bytes,
                                     hipStream_t hstream)
{
    return lic::call(args, workspace, workspace_bytes, hstream, false);
}

extern "C" int lic_attention_backward(const lic_attention_args *args, void *workspace, uint64_t workspace_bytes,
                                      hipStream_t hstream)
{
    return lic::call(args, workspace, workspace_bytes, hstream, true);
}
