// C entry points of kda_attention.h and kda_cache_q4.h: argument checks and dispatch.
#include <cmath>

#include "attn_checks.cuh"
#include "cache_q4.cuh"

namespace {

using namespace kda::host;

// An int32 array by name.
struct IntArray {
    const char* name;
    const int32_t* at;
    int64_t n;
};

// Every thread block of the plan reads all inputs while others write outputs.
kda_status_t check_plan_overlap(const kda_cache_plan_args& a) {
    const IntArray in[] = {{"cached_lens", a.cached_lens, a.n_seqs},
                           {"new_lens", a.new_lens, a.n_seqs},
                           {"free_blocks", a.free_blocks, a.n_free},
                           {"free_begin", a.free_begin, 1}};
    const IntArray out[] = {{"free_end", a.free_end, 1},
                            {"block_table", a.block_table, (int64_t)a.n_seqs * a.table_stride},
                            {"kv_lens", a.kv_lens, a.n_seqs},
                            {"cu_seqlens", a.cu_seqlens, (int64_t)a.n_seqs + 1},
                            {"slot_map", a.slot_map, a.max_tokens},
                            {"positions", a.positions, a.max_tokens}};
    for (const IntArray& x : in)
        for (const IntArray& y : out) {
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.at), y0 = reinterpret_cast<uintptr_t>(y.at);
            if (x.n > 0 && y.n > 0 && x0 < y0 + 4 * (uintptr_t)y.n && y0 < x0 + 4 * (uintptr_t)x.n)
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", y.name, x.name);
        }
    return KDA_OK;
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// How a suffix kernel divides its work: query heads of a unit, keys of a tile, workers of
// a thread block.
struct DecodeShape {
    int rows, tile, warps;
};
DecodeShape decode_shape(const kda_attn_decode_args& a) {
    return {kda::decode_rows(a.dtype, a.n_heads / a.n_kv_heads), kda::decode_tile(a.dtype, a.d), kda::kDecodeWarps};
}
DecodeShape decode_q4_shape(const kda_attn_decode_args& a) {
    const int G = a.n_heads / a.n_kv_heads;
    return {kda::q4_rows(a.dtype, G), kda::kQ4Keys, kda::q4_warps(kda::q4_columns(a.dtype, G))};
}

// Workers of the suffix kernel: all, or as many as the longest sequences that the
// table can name would give work.
int decode_pieces(const kda_attn_decode_args& a, const DecodeShape& shape) {
    const int64_t G = a.n_heads / a.n_kv_heads, all = 152 * (int64_t)shape.warps;
    const int64_t tiles = ((int64_t)a.table_stride * a.block_size + shape.tile - 1) / shape.tile;
    const int64_t units = (int64_t)a.n_seqs * a.n_kv_heads * ((G + shape.rows - 1) / shape.rows);
    const int least = kda::decode_least_tiles(tiles);
    if (tiles >= all * least) return (int)all;
    const int64_t pieces = (units * tiles / least + shape.warps) / shape.warps * shape.warps;
    return (int)(pieces < all ? pieces : all);
}

// What one more block of a shared prefix costs its rows' joins, in the unit of
// prefix_block_tiles.  Fitted to the best of 1 to 32 blocks for 8 to 300 sequences of 16
// and 40 heads behind 512 to 32768 positions (bf16, d = 128: 300 x 40 heads behind 512, one
// block 142 us and four 215 us; 8 x 40 heads behind 8192, one 110 us and eight 29 us.
// fp32: 83 x 16 behind 2048, one 288 us, eight 118 us, 32 170 us).
float prefix_split_cost(const kda_attn_decode_args& a) {
    return (a.dtype == KDA_BF16 ? 0.16f : 0.1f) * ((float)a.n_seqs * (float)a.n_heads + 300.f);
}

// Blocks of keys that a shared prefix is cut into at most: bf16 a thread block (256 rows)
// for each of 152 SMs, fp32 two (64 rows), no more than the longest prefix that the table
// can hold would be cut into, and 64.
int prefix_splits(const kda_attn_decode_args& a) {
    if (a.n_groups == 0) return 0;
    const bool bf16 = a.dtype == KDA_BF16;
    const int64_t G = a.n_heads / a.n_kv_heads;
    const int64_t items = ((int64_t)a.n_seqs * G / (bf16 ? 256 : 64) + a.n_groups) * a.n_kv_heads;
    const int64_t n = bf16 ? (152 + items - 1) / items : 304 / items;
    const int64_t most = 1 + (int64_t)sqrtf((float)a.table_stride * (float)a.block_size / prefix_split_cost(a));
    const int64_t r = n < most ? n : most;
    return (int)(r < 1 ? 1 : r > 64 ? 64 : r);
}

// Blocks of keys that a prompt's tiles are cut into: several where the row tiles (256
// rows in bf16, 64 in fp32) would leave most SMs idle and the keys are many.  The join and
// its launch cost about 5 us, so a block keeps 512 keys, or 640 of a packed bf16 prompt,
// whose rows see half of them on average.  bf16, d = 128: 16 queries behind 8192 positions,
// 8/2 heads, 25 us and 100 us uncut; one prompt of 8192, 2/1 heads, 64 and 95 us, of 2048,
// 4/1 heads, 23 and 29 us; of 1024, 8/8 heads, 20 us uncut and 25 us in two blocks.  fp32:
// 6 resumed prompts of one or two tokens behind up to 3776, 82 and 268 us; 1024 tokens of
// one head 25 and 35 us (2048 of two heads, where the tiles' own key groups would do, 78
// and 65 us).
int prompt_splits(const kda_attn_prefill_args& a) {
    if (a.n_seqs == 0 || a.total_tokens == 0) return 1;
    const bool bf16 = a.dtype == KDA_BF16;
    const int64_t G = a.n_heads / a.n_kv_heads;
    const int64_t items = (a.total_tokens * G / (bf16 ? 256 : 64) + a.n_seqs) * a.n_kv_heads;
    const int64_t keys = a.block_table ? (int64_t)a.table_stride * a.block_size : a.total_tokens;
    const int64_t n = 152 / items, most = keys / (bf16 && !a.block_table ? 640 : 512);
    const int64_t r = n < most ? n : most;
    return (int)(r < 2 ? 1 : r > 32 ? 32 : r);
}

size_t prompt_part_bytes(const kda_attn_prefill_args& a, int n) { return round_up((size_t)n * a.total_tokens * a.n_heads * a.d * sizeof(float)); }
size_t prompt_ml_bytes(const kda_attn_prefill_args& a, int n) { return round_up((size_t)n * a.total_tokens * a.n_heads * sizeof(float2)); }

struct DecodeSpace {
    size_t pre_o, pre_ml, part_o, part_ml, open, info, bytes;
};

DecodeSpace decode_space(const kda_attn_decode_args& a, const DecodeShape& shape) {
    DecodeSpace s{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += round_up(bytes);
        return r;
    };
    const size_t rows = (size_t)a.n_seqs * a.n_heads * prefix_splits(a);
    const size_t pieces = (size_t)decode_pieces(a, shape), parts = 2 * pieces * shape.rows;
    s.pre_o = take(rows * a.d * sizeof(float));
    s.pre_ml = take(rows * sizeof(float2));
    s.part_o = take(parts * a.d * sizeof(float));
    s.part_ml = take(parts * sizeof(float2));
    s.open = take(pieces * sizeof(int4));
    s.info = take(a.n_groups > 0 ? (size_t)a.n_seqs * sizeof(int2) : 0);
    s.bytes = at;
    return s;
}

kda_status_t check_decode_sizes(const kda_attn_decode_args& a) {
    KDA_TRY(check_heads(a.n_heads, a.n_kv_heads, a.d, a.dtype));
    KDA_TRY(check_seqs(a.n_seqs, "n_seqs"));
    KDA_TRY(check_seqs(a.n_groups, "n_groups"));
    KDA_TRY(check_block_size(a.block_size));
    KDA_TRY(check_table(a.table_stride, a.block_size));
    if ((int64_t)a.n_seqs * a.n_heads > (int64_t)INT32_MAX) return fail(KDA_ERR_INVALID_ARG, "n_seqs * n_heads too large");
    return KDA_OK;
}

kda_status_t check_prefill_sizes(const kda_attn_prefill_args& a) {
    KDA_TRY(check_heads(a.n_heads, a.n_kv_heads, a.d, a.dtype));
    KDA_TRY(check_seqs(a.n_seqs, "n_seqs"));
    KDA_TRY(check_scale(a.scale));
    if (a.total_tokens < 0 || a.total_tokens > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "total_tokens %lld outside [0, 2^31)", (long long)a.total_tokens);
    KDA_TRY(check_stride(a.q_stride, a.n_heads, a.d, a.dtype, "q_stride"));
    KDA_TRY(check_stride(a.o_stride, a.n_heads, a.d, a.dtype, "o_stride"));
    if (a.block_table) {
        KDA_TRY(check_block_size(a.block_size));
        KDA_TRY(check_table(a.table_stride, a.block_size));
        KDA_TRY(check_cache_size(a.n_blocks, a.block_size, a.n_kv_heads));
    } else {
        KDA_TRY(check_stride(a.k_stride, a.n_kv_heads, a.d, a.dtype, "k_stride"));
        KDA_TRY(check_stride(a.v_stride, a.n_kv_heads, a.d, a.dtype, "v_stride"));
    }
    // one thread block for each tile of at least one token
    if ((a.total_tokens + a.n_seqs) * 2 > (int64_t)INT32_MAX) return fail(KDA_ERR_INVALID_ARG, "total_tokens + n_seqs too large");
    return KDA_OK;
}

kda_status_t check_q4(const kda_cache_q4& c, int32_t n_kv_heads, bool used) {
    KDA_TRY(check_block_size(c.block_size));
    KDA_TRY(check_cache_size(c.n_blocks, c.block_size, n_kv_heads));
    if (c.reserved0 != 0) return fail(KDA_ERR_INVALID_ARG, "the cache's reserved0 must be 0");
    if (!used) return KDA_OK;
    KDA_TRY(check_ptr(c.k_codes, "k_codes"));
    KDA_TRY(check_ptr(c.k_scales, "k_scales"));
    KDA_TRY(check_ptr(c.v_codes, "v_codes"));
    return check_ptr(c.v_scales, "v_scales");
}

// An array by name.
struct Range {
    const char* name;
    const void* at;
    int64_t bytes;
};
struct Q4Ranges {
    Range at[4];
    Q4Ranges(const kda_cache_q4& c, int64_t n_kv_heads, int32_t d) {
        const int64_t rows = c.n_blocks * c.block_size * n_kv_heads, codes = rows * kda::q4_code_bytes(d), scales = rows * kda::q4_scale_bytes(d);
        at[0] = {"k_codes", c.k_codes, codes}, at[1] = {"v_codes", c.v_codes, codes};
        at[2] = {"k_scales", c.k_scales, scales}, at[3] = {"v_scales", c.v_scales, scales};
    }
};

kda_status_t check_append_q4_overlap(const kda_cache_append_q4_args& a) {
    const int64_t e = esize(a.dtype), width = a.n_kv_heads * (int64_t)a.d * e;
    auto rows = [&](const char* name, const void* at, int64_t stride) { return Range{name, at, at ? stride * e * (a.n_tokens - 1) + width : 0}; };
    const Range in[] = {rows("k", a.k, a.k_stride), rows("v", a.v, a.v_stride), {"slot_map", a.slot_map, 4 * a.n_tokens}};
    const Range out[] = {rows("k_out", a.k_out, a.k_out_stride), rows("v_out", a.v_out, a.v_out_stride)};
    const Q4Ranges cache(a.cache, a.n_kv_heads, a.d);
    for (int i = 0; i < 4; ++i) {
        for (const Range& x : in) KDA_TRY(check_ranges(cache.at[i].at, cache.at[i].bytes, cache.at[i].name, x.at, x.bytes, x.name));
        for (const Range& x : out) KDA_TRY(check_ranges(cache.at[i].at, cache.at[i].bytes, cache.at[i].name, x.at, x.bytes, x.name));
        for (int j = 0; j < i; ++j) KDA_TRY(check_ranges(cache.at[i].at, cache.at[i].bytes, cache.at[i].name, cache.at[j].at, cache.at[j].bytes, cache.at[j].name));
    }
    const int64_t in_stride[] = {a.k_stride * e, a.v_stride * e}, out_stride[] = {a.k_out_stride * e, a.v_out_stride * e};
    for (int i = 0; i < 2; ++i) {
        if (!out[i].at) continue;
        KDA_TRY(check_ranges(out[i].at, out[i].bytes, out[i].name, a.slot_map, 4 * a.n_tokens, "slot_map"));
        for (int j = 0; j < 2; ++j) {
            if (i == j && out[i].at == in[j].at && out_stride[i] == in_stride[j]) continue;
            if (tokens_overlap(out[i].at, out_stride[i], width, in[j].at, in_stride[j], width, a.n_tokens))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
        }
    }
    if (a.k_out && a.v_out && tokens_overlap(a.k_out, out_stride[0], width, a.v_out, out_stride[1], width, a.n_tokens))
        return fail(KDA_ERR_INVALID_ARG, "k_out overlaps v_out");
    return KDA_OK;
}

kda_status_t check_unpack_q4_overlap(const kda_cache_unpack_q4_args& a) {
    const int64_t bytes = a.n_blocks * a.cache.block_size * a.n_kv_heads * a.d * esize(a.dtype);
    const Q4Ranges cache(a.cache, a.n_kv_heads, a.d);
    const Range in[] = {cache.at[0], cache.at[1], cache.at[2], cache.at[3],
                        {"block_table", a.block_table, 4 * (int64_t)a.n_seqs * a.table_stride},
                        {"to_table", a.to_table, 4 * (int64_t)a.n_seqs * a.to_stride},
                        {"first", a.first, a.first ? 4 * (int64_t)a.n_seqs : 0},
                        {"kv_lens", a.kv_lens, 4 * (int64_t)a.n_seqs}};
    for (const Range& x : in) {
        KDA_TRY(check_ranges(a.k_cache, bytes, "k_cache", x.at, x.bytes, x.name));
        KDA_TRY(check_ranges(a.v_cache, bytes, "v_cache", x.at, x.bytes, x.name));
    }
    return check_ranges(a.k_cache, bytes, "k_cache", a.v_cache, bytes, "v_cache");
}

// The checks that decode attention over either cache makes; `wide`: whether k_cache, v_cache and
// n_blocks name a cache that is read.
kda_status_t check_decode(const kda_attn_decode_args& a, bool wide) {
    KDA_TRY(check_decode_sizes(a));
    KDA_TRY(check_scale(a.scale));
    if (a.reserved0 != 0) return fail(KDA_ERR_INVALID_ARG, "reserved0 must be 0");
    if (wide) KDA_TRY(check_cache_size(a.n_blocks, a.block_size, a.n_kv_heads));
    KDA_TRY(check_stride(a.q_stride, a.n_heads, a.d, a.dtype, "q_stride"));
    KDA_TRY(check_stride(a.o_stride, a.n_heads, a.d, a.dtype, "o_stride"));
    if (a.n_seqs == 0) return KDA_OK;
    KDA_TRY(check_ptr(a.q, "q"));
    KDA_TRY(check_ptr(a.o, "o"));
    if (wide) {
        KDA_TRY(check_ptr(a.k_cache, "k_cache"));
        KDA_TRY(check_ptr(a.v_cache, "v_cache"));
    }
    KDA_TRY(check_int(a.block_table, "block_table"));
    KDA_TRY(check_int(a.kv_lens, "kv_lens"));
    if (a.lse) KDA_TRY(check_int(a.lse, "lse"));
    if (a.n_groups > 0) {
        KDA_TRY(check_int(a.group_start, "group_start"));
        KDA_TRY(check_int(a.prefix_lens, "prefix_lens"));
    }
    return KDA_OK;
}

// Lays out the workspace in *out and starts what comes before the suffixes: the shared prefixes.
kda_status_t start_decode(const kda_attn_decode_args& a, const DecodeShape& shape, cudaStream_t s, kda::AttnDecodeLaunch* out) {
    const DecodeSpace sp = decode_space(a, shape);
    if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u))
        return fail(KDA_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (a.workspace_bytes < sp.bytes)
        return fail(KDA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", a.workspace_bytes, sp.bytes);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    kda::AttnDecodeLaunch& p = *out;
    p = kda::AttnDecodeLaunch{};
    p.a = a;
    p.n_pieces = decode_pieces(a, shape);
    p.n_split = prefix_splits(a);
    p.split_cost = prefix_split_cost(a);
    p.prefix_tile = a.dtype == KDA_BF16 ? kda::kTileKeysBf16 : kda::kTileKeysF32;
    p.pre_o = reinterpret_cast<float*>(ws + sp.pre_o);
    p.pre_ml = reinterpret_cast<float2*>(ws + sp.pre_ml);
    p.part_o = reinterpret_cast<float*>(ws + sp.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + sp.part_ml);
    p.open = reinterpret_cast<int4*>(ws + sp.open);
    p.info = reinterpret_cast<int2*>(ws + sp.info);
    KDA_TRY(kda::device_status_word(&p.status));
    if (a.n_groups > 0) {
        cudaError_t e = kda::launch_decode_info(p, s);
        if (e != cudaSuccess) return cuda_fail(e, "decode plan launch");
        kda::AttnTileLaunch t{};
        t.a.n_seqs = a.n_groups;
        t.a.n_heads = a.n_heads, t.a.n_kv_heads = a.n_kv_heads, t.a.d = a.d, t.a.dtype = a.dtype;
        t.a.scale = a.scale;
        t.a.total_tokens = a.n_seqs;
        t.a.q_stride = a.q_stride;
        t.a.q = a.q;
        t.a.cu_seqlens = a.group_start;
        t.a.k_cache = a.k_cache, t.a.v_cache = a.v_cache;
        t.a.block_table = a.block_table;
        t.a.n_blocks = a.n_blocks, t.a.block_size = a.block_size, t.a.table_stride = a.table_stride;
        t.status = p.status;
        t.prefix_lens = a.prefix_lens;
        t.n_split = p.n_split;
        t.split_cost = p.split_cost;
        t.part_o = p.pre_o;
        t.part_ml = p.pre_ml;
        e = kda::launch_attn_tile(t, s);
        if (e != cudaSuccess) return cuda_fail(e, "shared-prefix attention launch");
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_cache_plan(const kda_cache_plan_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_cache_plan_args& a = *args;
    KDA_TRY(check_seqs(a.n_seqs, "n_seqs"));
    KDA_TRY(check_block_size(a.block_size));
    KDA_TRY(check_table(a.table_stride, a.block_size));
    KDA_TRY(check_cache_size(a.n_blocks, a.block_size, 1));
    if (a.n_free < 0) return fail(KDA_ERR_INVALID_ARG, "n_free < 0");
    if (a.max_tokens < 0 || a.max_tokens > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "max_tokens %lld outside [0, 2^31)", (long long)a.max_tokens);
    KDA_TRY(check_int(a.free_begin, "free_begin"));
    KDA_TRY(check_int(a.free_end, "free_end"));
    if (a.free_begin == a.free_end) return fail(KDA_ERR_INVALID_ARG, "free_begin and free_end must differ");
    if (a.n_free > 0) KDA_TRY(check_int(a.free_blocks, "free_blocks"));
    KDA_TRY(check_int(a.cu_seqlens, "cu_seqlens"));
    if (a.n_seqs > 0) {
        KDA_TRY(check_int(a.cached_lens, "cached_lens"));
        KDA_TRY(check_int(a.new_lens, "new_lens"));
        KDA_TRY(check_int(a.block_table, "block_table"));
        KDA_TRY(check_int(a.kv_lens, "kv_lens"));
    }
    if (a.max_tokens > 0) {
        KDA_TRY(check_int(a.slot_map, "slot_map"));
        KDA_TRY(check_int(a.positions, "positions"));
    }
    KDA_TRY(check_plan_overlap(a));
    kda::CachePlanLaunch p{a, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_cache_plan(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "cache plan launch");
}

kda_status_t kda_cache_append(int64_t n_tokens, int32_t n_kv_heads, int32_t d, int32_t dtype, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slot_map,
                              void* k_cache, void* v_cache, int64_t n_blocks, int32_t block_size, void* stream) {
    KDA_TRY(check_heads(n_kv_heads, n_kv_heads, d, dtype));
    KDA_TRY(check_block_size(block_size));
    KDA_TRY(check_cache_size(n_blocks, block_size, n_kv_heads));
    KDA_TRY(check_stride(k_stride, n_kv_heads, d, dtype, "k_stride"));
    KDA_TRY(check_stride(v_stride, n_kv_heads, d, dtype, "v_stride"));
    if (n_tokens < 0 || n_tokens > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "n_tokens %lld outside [0, 2^31)", (long long)n_tokens);
    if (n_tokens == 0) return KDA_OK;
    KDA_TRY(check_ptr(k, "k"));
    KDA_TRY(check_ptr(v, "v"));
    KDA_TRY(check_int(slot_map, "slot_map"));
    KDA_TRY(check_ptr(k_cache, "k_cache"));
    KDA_TRY(check_ptr(v_cache, "v_cache"));
    const int vec = 16 / esize(dtype);
    kda::CacheAppendLaunch p{n_tokens, n_kv_heads, n_kv_heads * (d / vec), d / vec, k, v, k_stride / vec, v_stride / vec,
                             slot_map, k_cache, v_cache, n_blocks, block_size, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_cache_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "cache append launch");
}

size_t kda_attn_prefill_workspace_size(const kda_attn_prefill_args* args) {
    if (!args || check_prefill_sizes(*args) != KDA_OK) return 0;
    const int n = prompt_splits(*args);
    return n > 1 ? prompt_part_bytes(*args, n) + prompt_ml_bytes(*args, n) : 0;
}

kda_status_t kda_attn_prefill(const kda_attn_prefill_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_attn_prefill_args& a = *args;
    KDA_TRY(check_prefill_sizes(a));
    if (a.n_seqs == 0 || a.total_tokens == 0) return KDA_OK;
    KDA_TRY(check_ptr(a.q, "q"));
    KDA_TRY(check_ptr(a.o, "o"));
    KDA_TRY(check_int(a.cu_seqlens, "cu_seqlens"));
    if (a.lse) KDA_TRY(check_int(a.lse, "lse"));
    if (a.block_table) {
        KDA_TRY(check_ptr(a.k_cache, "k_cache"));
        KDA_TRY(check_ptr(a.v_cache, "v_cache"));
        KDA_TRY(check_int(a.block_table, "block_table"));
        KDA_TRY(check_int(a.kv_lens, "kv_lens"));
    } else {
        KDA_TRY(check_ptr(a.k, "k"));
        KDA_TRY(check_ptr(a.v, "v"));
    }
    kda::AttnTileLaunch p{a, nullptr, nullptr, 1, 0.f, nullptr, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n = prompt_splits(a);
    if (n > 1 && a.workspace && a.workspace_bytes >= prompt_part_bytes(a, n) + prompt_ml_bytes(a, n)) {
        if (reinterpret_cast<uintptr_t>(a.workspace) & 255u) return fail(KDA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        p.n_split = n;
        p.part_o = static_cast<float*>(a.workspace);
        p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) + prompt_part_bytes(a, n));
        const cudaError_t e = cudaMemsetAsync(p.part_ml, kda::kUnwritten, (size_t)a.total_tokens * a.n_heads * sizeof(float2), s);
        if (e != cudaSuccess) return cuda_fail(e, "prompt attention workspace");
    }
    cudaError_t e = kda::launch_attn_tile(p, s);
    if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
    if (p.n_split > 1) e = kda::launch_prompt_join(p, s);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "prompt attention join launch");
}

size_t kda_attn_decode_workspace_size(const kda_attn_decode_args* args) {
    if (!args || check_decode_sizes(*args) != KDA_OK || args->n_seqs == 0) return 0;
    return decode_space(*args, decode_shape(*args)).bytes;
}

kda_status_t kda_attn_decode(const kda_attn_decode_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_attn_decode_args& a = *args;
    KDA_TRY(check_decode(a, true));
    if (a.n_seqs == 0) return KDA_OK;
    kda::AttnDecodeLaunch p;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    KDA_TRY(start_decode(a, decode_shape(a), s, &p));
    const cudaError_t e = a.dtype == KDA_BF16 ? kda::launch_decode_mma(p, s) : kda::launch_decode_simt(p, s);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "decode attention launch");
}

size_t kda_attn_decode_q4_workspace_size(const kda_attn_decode_q4_args* args) {
    if (!args || check_decode_sizes(args->base) != KDA_OK || args->base.n_seqs == 0) return 0;
    return decode_space(args->base, decode_q4_shape(args->base)).bytes;
}

kda_status_t kda_attn_decode_q4(const kda_attn_decode_q4_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_attn_decode_args& a = args->base;
    KDA_TRY(check_decode(a, a.n_groups > 0));
    KDA_TRY(check_q4(args->cache, a.n_kv_heads, a.n_seqs > 0));
    if (args->cache.block_size != a.block_size)
        return fail(KDA_ERR_INVALID_ARG, "the cache's block_size %d and base.block_size %d differ", args->cache.block_size, a.block_size);
    if (a.n_seqs == 0) return KDA_OK;
    kda::AttnDecodeQ4Launch p;
    p.cache = args->cache;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    KDA_TRY(start_decode(a, decode_q4_shape(a), s, &p.base));
    const cudaError_t e = kda::launch_decode_q4(p, s);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "4-bit decode attention launch");
}

kda_status_t kda_cache_append_q4(const kda_cache_append_q4_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_cache_append_q4_args& a = *args;
    KDA_TRY(check_heads(a.n_kv_heads, a.n_kv_heads, a.d, a.dtype));
    if (a.reserved0 != 0) return fail(KDA_ERR_INVALID_ARG, "reserved0 must be 0");
    KDA_TRY(check_stride(a.k_stride, a.n_kv_heads, a.d, a.dtype, "k_stride"));
    KDA_TRY(check_stride(a.v_stride, a.n_kv_heads, a.d, a.dtype, "v_stride"));
    if (a.k_out) KDA_TRY(check_stride(a.k_out_stride, a.n_kv_heads, a.d, a.dtype, "k_out_stride"));
    if (a.v_out) KDA_TRY(check_stride(a.v_out_stride, a.n_kv_heads, a.d, a.dtype, "v_out_stride"));
    if (a.n_tokens < 0 || a.n_tokens > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "n_tokens %lld outside [0, 2^31)", (long long)a.n_tokens);
    KDA_TRY(check_q4(a.cache, a.n_kv_heads, a.n_tokens > 0));
    if (a.n_tokens == 0) return KDA_OK;
    KDA_TRY(check_ptr(a.k, "k"));
    KDA_TRY(check_ptr(a.v, "v"));
    KDA_TRY(check_int(a.slot_map, "slot_map"));
    if (a.k_out) KDA_TRY(check_ptr(a.k_out, "k_out"));
    if (a.v_out) KDA_TRY(check_ptr(a.v_out, "v_out"));
    KDA_TRY(check_append_q4_overlap(a));
    kda::CacheAppendQ4Launch p{a, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_append_q4(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "4-bit append launch");
}

kda_status_t kda_cache_unpack_q4(const kda_cache_unpack_q4_args* args, void* stream) {
    if (!args) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_cache_unpack_q4_args& a = *args;
    KDA_TRY(check_heads(a.n_kv_heads, a.n_kv_heads, a.d, a.dtype));
    KDA_TRY(check_seqs(a.n_seqs, "n_seqs"));
    KDA_TRY(check_q4(a.cache, a.n_kv_heads, a.n_seqs > 0));
    KDA_TRY(check_table(a.table_stride, a.cache.block_size));
    KDA_TRY(check_table(a.to_stride, a.cache.block_size));
    KDA_TRY(check_cache_size(a.n_blocks, a.cache.block_size, a.n_kv_heads));
    if (a.n_seqs == 0) return KDA_OK;
    KDA_TRY(check_int(a.block_table, "block_table"));
    KDA_TRY(check_int(a.to_table, "to_table"));
    if (a.first) KDA_TRY(check_int(a.first, "first"));
    KDA_TRY(check_int(a.kv_lens, "kv_lens"));
    KDA_TRY(check_ptr(a.k_cache, "k_cache"));
    KDA_TRY(check_ptr(a.v_cache, "v_cache"));
    KDA_TRY(check_unpack_q4_overlap(a));
    kda::CacheUnpackQ4Launch p{a, nullptr};
    KDA_TRY(kda::device_status_word(&p.status));
    const cudaError_t e = kda::launch_unpack_q4(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "4-bit read-back launch");
}

}  // extern "C"
