// Argument checks shared by the C entry points of the softmax-attention side (host code).
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "attn_common.cuh"

namespace kda {
namespace host {

__attribute__((format(printf, 2, 3))) inline kda_status_t fail(kda_status_t st, const char* fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return kda::record_error(st, text);
}

inline kda_status_t cuda_fail(cudaError_t e, const char* what) {
    return fail(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define KDA_TRY(call)                       \
    do {                                    \
        const kda_status_t st_ = (call);    \
        if (st_ != KDA_OK) return st_;      \
    } while (0)

inline kda_status_t check_ptr(const void* p, const char* name) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 15u) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}

// Single integers need only their own alignment.
inline kda_status_t check_int(const void* p, const char* name) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(KDA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return KDA_OK;
}

constexpr int64_t kMaxSeqs = 1 << 20;
constexpr int64_t kMaxHeads = 4096, kMaxGroup = 128;

inline kda_status_t check_heads(int32_t H, int32_t H_kv, int32_t d, int32_t dtype) {
    if (H_kv <= 0 || H <= 0 || H % H_kv) return fail(KDA_ERR_INVALID_ARG, "n_heads %d must be a positive multiple of n_kv_heads %d", H, H_kv);
    if (H > kMaxHeads || H / H_kv > kMaxGroup)
        return fail(KDA_ERR_UNSUPPORTED, "at most %d heads and %d query heads per key/value head (got %d, %d)", (int)kMaxHeads, (int)kMaxGroup, H, H / H_kv);
    if (d != 64 && d != 128) return fail(KDA_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d);
    if (dtype != KDA_BF16 && dtype != KDA_FP32) return fail(KDA_ERR_UNSUPPORTED, "dtype %d", dtype);
    return KDA_OK;
}

inline int esize(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }

inline kda_status_t check_stride(int64_t stride, int64_t heads, int32_t d, int32_t dtype, const char* name) {
    if (stride < heads * d || stride * esize(dtype) % 16 || stride > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "%s %lld must be a multiple of 16 bytes, at least %lld and below 2^31", name,
                    (long long)stride, (long long)heads * d);
    return KDA_OK;
}

inline kda_status_t check_block_size(int32_t bs) {
    if (bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256)
        return fail(KDA_ERR_UNSUPPORTED, "block_size must be 16, 32, 64, 128 or 256 (got %d)", bs);
    return KDA_OK;
}

inline kda_status_t check_cache_size(int64_t n_blocks, int32_t bs, int32_t H_kv) {
    if (n_blocks <= 0 || n_blocks > (int64_t)INT32_MAX / ((int64_t)bs * H_kv))
        return fail(KDA_ERR_INVALID_ARG, "n_blocks %lld must be positive, with n_blocks * block_size * n_kv_heads < 2^31", (long long)n_blocks);
    return KDA_OK;
}

inline kda_status_t check_seqs(int32_t n, const char* name) {
    if (n < 0 || n > kMaxSeqs) return fail(KDA_ERR_INVALID_ARG, "%s %d outside [0, %lld]", name, n, (long long)kMaxSeqs);
    return KDA_OK;
}

inline kda_status_t check_table(int32_t stride, int32_t bs) {
    if (stride < 1 || (int64_t)stride * bs > (int64_t)INT32_MAX)
        return fail(KDA_ERR_INVALID_ARG, "table_stride %d must be positive, with table_stride * block_size < 2^31", stride);
    return KDA_OK;
}

inline kda_status_t check_scale(float scale) {
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    return KDA_OK;
}

// Whether two arrays of `bytes` share one.
inline kda_status_t check_ranges(const void* out, int64_t out_bytes, const char* out_name, const void* x, int64_t x_bytes, const char* name) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(x);
    if (out_bytes > 0 && x_bytes > 0 && a < b + (uintptr_t)x_bytes && b < a + (uintptr_t)out_bytes)
        return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", out_name, name);
    return KDA_OK;
}

// Whether two tensors of n tokens (each `width` bytes, `stride` bytes apart) share a byte.  Views
// of one projection's output have one stride and lie beside each other in each token; tensors of
// different strides whose ranges meet count as overlapping.
inline bool tokens_overlap(const void* x, int64_t x_stride, int64_t x_width, const void* y, int64_t y_stride, int64_t y_width, int64_t n) {
    const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(x), b = (int64_t)reinterpret_cast<uintptr_t>(y);
    if (a + x_stride * (n - 1) + x_width <= b || b + y_stride * (n - 1) + y_width <= a) return false;
    if (n == 1) return true;
    if (x_stride != y_stride) return true;
    const int64_t apart = ((b - a) % x_stride + x_stride) % x_stride;    // y's start within x's token, or before the next
    return apart < x_width || apart + y_width > x_stride;
}

}  // namespace host
}  // namespace kda
