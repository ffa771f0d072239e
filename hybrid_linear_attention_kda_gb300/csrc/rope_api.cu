// C entry points of kda_rope.h: argument checks and dispatch.
#include "attn_checks.cuh"
#include "rope.cuh"

namespace {

using namespace kda::host;

// A tensor [T, heads, d] by name.
struct Rows {
    const char* name;
    const void* at;
    int64_t stride;              // bytes
    int64_t width;               // bytes of a token
    int64_t n;
};

kda_status_t check_apart(const Rows& out, const Rows& other) {
    if (!tokens_overlap(out.at, out.stride, out.width, other.at, other.stride, other.width, out.n)) return KDA_OK;
    return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", out.name, other.name);
}

// What an output may not share with the tensor it is made of, unless it is that tensor.
kda_status_t check_apart_or_same(const Rows& out, const Rows& from) {
    return out.at == from.at && out.stride == from.stride ? KDA_OK : check_apart(out, from);
}

kda_status_t check_sizes(const kda_qk_rope_args& a, bool append) {
    if (a.n_tokens < 0 || a.n_tokens > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "n_tokens %lld outside [0, 2^31)", (long long)a.n_tokens);
    KDA_TRY(check_heads(a.n_kv_heads, a.n_kv_heads, a.d, a.dtype));
    const bool queries = !append || a.n_heads != 0;
    if (queries) KDA_TRY(check_heads(a.n_heads, a.n_heads, a.d, a.dtype));
    else if (a.q || a.q_out || a.q_weight) return fail(KDA_ERR_INVALID_ARG, "q, q_out and q_weight must be NULL where n_heads is 0");
    if (a.rot_dim < 0 || a.rot_dim > a.d || a.rot_dim % 8)
        return fail(KDA_ERR_INVALID_ARG, "rot_dim %d must be a multiple of 8 in [0, d]", a.rot_dim);
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (a.interleaved != 0 && a.interleaved != 1) return fail(KDA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (a.reserved0 != 0) return fail(KDA_ERR_INVALID_ARG, "reserved0 must be 0");
    if (queries) {
        KDA_TRY(check_stride(a.q_stride, a.n_heads, a.d, a.dtype, "q_stride"));
        KDA_TRY(check_stride(a.q_out_stride, a.n_heads, a.d, a.dtype, "q_out_stride"));
    }
    KDA_TRY(check_stride(a.k_stride, a.n_kv_heads, a.d, a.dtype, "k_stride"));
    if (!append) KDA_TRY(check_stride(a.k_out_stride, a.n_kv_heads, a.d, a.dtype, "k_out_stride"));
    return KDA_OK;
}

kda_status_t check_pointers(const kda_qk_rope_args& a) {
    if (a.n_heads) {
        KDA_TRY(check_ptr(a.q, "q"));
        KDA_TRY(check_ptr(a.q_out, "q_out"));
    }
    KDA_TRY(check_ptr(a.k, "k"));
    if (a.q_weight) KDA_TRY(check_ptr(a.q_weight, "q_weight"));
    if (a.k_weight) KDA_TRY(check_ptr(a.k_weight, "k_weight"));
    if (a.rot_dim) KDA_TRY(check_ptr(a.turns, "turns"));
    return check_int(a.positions, "positions");
}

Rows rows(const char* name, const void* at, int64_t stride, int64_t heads, const kda_qk_rope_args& a) {
    return {name, at, stride * esize(a.dtype), heads * a.d * esize(a.dtype), a.n_tokens};
}

// A dense array as rows without an end to end gap.
Rows whole(const char* name, const void* at, int64_t bytes) { return {name, at, bytes, bytes, 1}; }

// No output may overlap what every row reads.
kda_status_t check_shared_inputs(const Rows& out, const kda_qk_rope_args& a) {
    const Rows shared[] = {whole("positions", a.positions, 4 * a.n_tokens), whole("turns", a.turns, 4 * a.rot_dim),
                           whole("q_weight", a.q_weight, a.q_weight ? 4 * a.d : 0), whole("k_weight", a.k_weight, a.k_weight ? 4 * a.d : 0)};
    for (const Rows& x : shared) KDA_TRY(check_ranges(out.at, out.stride * (out.n - 1) + out.width, out.name, x.at, x.width, x.name));
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_qk_norm_rope(const kda_qk_rope_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_qk_rope_args& a = *args;
    KDA_TRY(check_sizes(a, false));
    if (a.n_tokens == 0) return KDA_OK;
    KDA_TRY(check_pointers(a));
    KDA_TRY(check_ptr(a.k_out, "k_out"));
    const Rows q = rows("q", a.q, a.q_stride, a.n_heads, a), k = rows("k", a.k, a.k_stride, a.n_kv_heads, a);
    const Rows q_out = rows("q_out", a.q_out, a.q_out_stride, a.n_heads, a), k_out = rows("k_out", a.k_out, a.k_out_stride, a.n_kv_heads, a);
    KDA_TRY(check_apart_or_same(q_out, q));
    KDA_TRY(check_apart_or_same(k_out, k));
    KDA_TRY(check_apart(q_out, k));
    KDA_TRY(check_apart(k_out, q));
    KDA_TRY(check_apart(q_out, k_out));
    KDA_TRY(check_shared_inputs(q_out, a));
    KDA_TRY(check_shared_inputs(k_out, a));
    kda::RopeLaunch p{};
    p.a = a;
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_rope(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "norm and rotation launch");
}

kda_status_t kda_cache_append_rope(const kda_cache_append_rope_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_qk_rope_args& a = args->qk;
    KDA_TRY(check_sizes(a, true));
    KDA_TRY(check_stride(args->v_stride, a.n_kv_heads, a.d, a.dtype, "v_stride"));
    KDA_TRY(check_block_size(args->block_size));
    KDA_TRY(check_cache_size(args->n_blocks, args->block_size, a.n_kv_heads));
    if (args->reserved0 != 0) return fail(KDA_ERR_INVALID_ARG, "reserved0 must be 0");
    if (a.n_tokens == 0) return KDA_OK;
    KDA_TRY(check_pointers(a));
    KDA_TRY(check_ptr(args->v, "v"));
    KDA_TRY(check_int(args->slot_map, "slot_map"));
    KDA_TRY(check_ptr(args->k_cache, "k_cache"));
    KDA_TRY(check_ptr(args->v_cache, "v_cache"));
    const Rows in[] = {rows("q", a.q, a.q_stride, a.n_heads, a), rows("k", a.k, a.k_stride, a.n_kv_heads, a),
                       rows("v", args->v, args->v_stride, a.n_kv_heads, a)};
    const int64_t cache_bytes = args->n_blocks * a.n_kv_heads * args->block_size * a.d * esize(a.dtype);
    const Rows q_out = rows("q_out", a.q_out, a.q_out_stride, a.n_heads, a);
    const Rows k_cache = whole("k_cache", args->k_cache, cache_bytes), v_cache = whole("v_cache", args->v_cache, cache_bytes);
    KDA_TRY(check_ranges(k_cache.at, cache_bytes, "k_cache", v_cache.at, cache_bytes, "v_cache"));
    for (const Rows& cache : {k_cache, v_cache}) {
        for (const Rows& x : in)
            if (x.width) KDA_TRY(check_ranges(cache.at, cache_bytes, cache.name, x.at, x.stride * (x.n - 1) + x.width, x.name));
        KDA_TRY(check_shared_inputs(cache, a));
        KDA_TRY(check_ranges(cache.at, cache_bytes, cache.name, args->slot_map, 4 * a.n_tokens, "slot_map"));
    }
    if (a.n_heads) {
        KDA_TRY(check_apart_or_same(q_out, in[0]));
        KDA_TRY(check_apart(q_out, in[1]));
        KDA_TRY(check_apart(q_out, in[2]));
        KDA_TRY(check_shared_inputs(q_out, a));
        const int64_t q_bytes = q_out.stride * (q_out.n - 1) + q_out.width;
        KDA_TRY(check_ranges(q_out.at, q_bytes, "q_out", args->slot_map, 4 * a.n_tokens, "slot_map"));
        KDA_TRY(check_ranges(q_out.at, q_bytes, "q_out", k_cache.at, cache_bytes, "k_cache"));
        KDA_TRY(check_ranges(q_out.at, q_bytes, "q_out", v_cache.at, cache_bytes, "v_cache"));
    }
    kda::RopeLaunch p{a, true, args->v, args->v_stride, args->slot_map, args->k_cache, args->v_cache, args->n_blocks, args->block_size, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_rope(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "rotated append launch");
}

}  // extern "C"
