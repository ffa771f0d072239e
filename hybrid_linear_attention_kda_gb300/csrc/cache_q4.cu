// The 4-bit paged cache: append and read-back (include/kda_cache_q4.h has the format).
#include <float.h>
#include <math_constants.h>

#include "cache_q4.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// x rounded to bf16 towards -inf, towards +inf (x >= 0), as a float.
__device__ __forceinline__ float bf16_down(float x) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float((b + (b >> 31 ? 0xFFFFu : 0u)) & 0xFFFF0000u);
}
__device__ __forceinline__ float bf16_up(float x) { return __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u); }

// Eight channels as they lie in memory.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void open(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    __device__ __forceinline__ void close(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<float> {
    float4 r[2];
    __device__ __forceinline__ void open(float (&x)[8]) const {
        x[0] = r[0].x, x[1] = r[0].y, x[2] = r[0].z, x[3] = r[0].w;
        x[4] = r[1].x, x[5] = r[1].y, x[6] = r[1].z, x[7] = r[1].w;
    }
    __device__ __forceinline__ void close(const float (&x)[8]) {
        r[0] = make_float4(x[0], x[1], x[2], x[3]);
        r[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

constexpr int kAppendVecs = 2;

// A thread takes eight channels, eight lanes a group.  A thread block takes whole tokens (k
// and v, all heads): block_tokens of them.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ CacheAppendQ4Launch p, int32_t block_tokens) {
    griddep_wait();
    const kda_cache_append_q4_args& a = p.a;
    const uint32_t head_vecs = (uint32_t)a.d / 8, row_vecs = head_vecs * (uint32_t)a.n_kv_heads, page = (uint32_t)a.cache.block_size;
    const int64_t t0 = (int64_t)blockIdx.x * block_tokens, n_slots = a.cache.n_blocks * a.cache.block_size;
    const uint32_t n = 2 * row_vecs * (uint32_t)min((int64_t)block_tokens, a.n_tokens - t0);
    const int lane = threadIdx.x & 31;
    for (uint32_t base = 0; base < n; base += kThreads * kAppendVecs) {
        Eight<T> in[kAppendVecs];
        int32_t slot[kAppendVecs];
#pragma unroll
        for (int m = 0; m < kAppendVecs; ++m) {
            const uint32_t i = base + m * kThreads + threadIdx.x;
            in[m] = Eight<T>{};
            slot[m] = -1;
            if (i >= n) continue;
            const uint32_t half = i / row_vecs, x = i - half * row_vecs;     // half: 2 * token, or that + 1 for v
            const int64_t t = t0 + (half >> 1);
            slot[m] = a.slot_map[t];
            const T* from = static_cast<const T*>(half & 1 ? a.v : a.k) + t * (half & 1 ? a.v_stride : a.k_stride) + x * 8;
            in[m] = *reinterpret_cast<const Eight<T>*>(from);
        }
#pragma unroll
        for (int m = 0; m < kAppendVecs; ++m) {
            const uint32_t i = base + m * kThreads + threadIdx.x;
            float x[8];
            in[m].open(x);
            float lo = x[0], hi = x[0];
            bool odd = false;                                // something is not finite
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo = fminf(lo, x[e]), hi = fmaxf(hi, x[e]);
                odd |= !(fabsf(x[e]) <= FLT_MAX);
            }
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
            }
            const uint32_t odd_lanes = __ballot_sync(0xffffffffu, odd) >> (lane & 24) & 0xFFu;
            float low = bf16_down(lo), step = bf16_up(__fdiv_rn(__fsub_rn(hi, low), 15.f));
            const bool fine = !odd_lanes && low >= -FLT_MAX && __fsub_rn(hi, low) <= FLT_MAX && step <= FLT_MAX;
            if (!fine) low = CUDART_NAN_F, step = 0.f;
            uint32_t codes = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t code = 0;
                if (step > 0.f) code = min(__float2uint_rn(__fdiv_rn(__fsub_rn(x[e], low), step)), 15u);
                codes |= code << (4 * e);
                x[e] = fmaf((float)code, step, low);
            }
            if (slot[m] < 0 || slot[m] >= n_slots) {
                if (slot[m] != -1) flag(p.status, KDA_DEV_BAD_SLOT);
                continue;
            }
            const uint32_t half = i / row_vecs, y = i - half * row_vecs, h = y / head_vecs, e = y - h * head_vecs;
            const bool is_v = half & 1;
            const uint32_t block = (uint32_t)slot[m] / page, off = (uint32_t)slot[m] - block * page;
            const int64_t row = ((int64_t)block * a.n_kv_heads + h) * page + off;
            static_cast<uint32_t*>(is_v ? a.cache.v_codes : a.cache.k_codes)[row * head_vecs + e] = codes;
            if (e % 8 == 0)
                static_cast<uint32_t*>(is_v ? a.cache.v_scales : a.cache.k_scales)[row * (head_vecs / 8) + e / 8] =
                    __float_as_uint(step) >> 16 | (__float_as_uint(low) & 0xFFFF0000u);
            void* out = is_v ? a.v_out : a.k_out;
            if (out) {
                in[m].close(x);
                *reinterpret_cast<Eight<T>*>(static_cast<T*>(out) + (t0 + (half >> 1)) * (is_v ? a.v_out_stride : a.k_out_stride) + y * 8) = in[m];
            }
        }
    }
}

// ------------------------------------------------------------------ read-back

constexpr int kWarps = kThreads / 32, kRows = 16;           // an item: 16 positions of one head

// Eight values of codes w, as T.
template <typename T> __device__ __forceinline__ void write_eight(T* to, uint32_t w, float step, float low) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf((float)(w >> (4 * e) & 15u), step, low);
    Eight<T> v;
    v.close(x);
    *reinterpret_cast<Eight<T>*>(to) = v;
}

// Items in the order of sequences, positions, heads, dealt to the warps in turn, so that all
// warps work side by side whatever the lengths are.  Every thread block runs the (short)
// scan over the sequences itself.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_q4_kernel(const __grid_constant__ CacheUnpackQ4Launch p) {
    griddep_wait();
    __shared__ int64_t scan_buf[kWarps];
    __shared__ int64_t s_end[kThreads];
    __shared__ int2 s_range[kThreads];                       // positions from, to
    const kda_cache_unpack_q4_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, bs = a.cache.block_size, shift = __ffs(bs) - 1;
    constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes, kSteps = kRows / kAtOnce;    // lanes of a row, rows of a step
    const int own_row = lane / kLanes, own = lane % kLanes;
    const int64_t cap = (int64_t)min(a.table_stride, a.to_stride) * bs;
    const int64_t workers = (int64_t)gridDim.x * kWarps, worker = (int64_t)blockIdx.x * kWarps + (tid >> 5);
    int64_t base = 0;                                        // items of the sequences before this chunk
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
        const int32_t s = s0 + tid;
        int64_t items = 0;
        int2 range = make_int2(0, 0);
        if (s < a.n_seqs) {
            const int64_t kv = a.kv_lens[s];
            const int32_t first = a.first ? a.first[s] : 0;
            if (kv < 0 || kv > cap || first < 0) {
                if (blockIdx.x == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
            } else if (first < kv) {
                range = make_int2(first, (int)kv);
                items = ((kv + kRows - 1) / kRows - first / kRows) * a.n_kv_heads;
            }
        }
        int64_t total;
        s_end[tid] = block_scan<kThreads>(items, scan_buf, &total);
        s_range[tid] = range;
        __syncthreads();
        int64_t x = worker - base % workers;                 // the chunk's items that are this warp's
        if (x < 0) x += workers;
        for (; x < total; x += workers) {
            int i = 0;                                       // the first sequence that ends behind x
#pragma unroll
            for (int step = kThreads / 2; step > 0; step >>= 1)
                if (s_end[i + step - 1] <= x) i += step;
            const int64_t rel = x - (i ? s_end[i - 1] : 0);
            const int2 r = s_range[i];
            const int32_t piece = (int32_t)(rel / a.n_kv_heads), h = (int32_t)(rel - (int64_t)piece * a.n_kv_heads);
            const int32_t pos0 = (r.x / kRows + piece) * kRows, j = pos0 >> shift;
            const int32_t from = a.block_table[(int64_t)(s0 + i) * a.table_stride + j];
            const int32_t to = a.to_table[(int64_t)(s0 + i) * a.to_stride + j];
            if (from < 0 || from >= a.cache.n_blocks || to < 0 || to >= a.n_blocks) {
                if (lane == 0) flag(p.status, KDA_DEV_BAD_SLOT);
                continue;
            }
            const int64_t src = ((int64_t)from * a.n_kv_heads + h) * bs + (pos0 & (bs - 1)) + own_row;
            const int64_t dst = ((int64_t)to * a.n_kv_heads + h) * bs + (pos0 & (bs - 1)) + own_row;
            uint2 codes[2][kSteps];
            uint32_t scale[2][kSteps];
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int64_t row = src + k * kAtOnce;
                    codes[v][k] = static_cast<const uint2*>(v ? a.cache.v_codes : a.cache.k_codes)[row * kLanes + own];
                    scale[v][k] = static_cast<const uint32_t*>(v ? a.cache.v_scales : a.cache.k_scales)[row * (D / kQ4Group) + own / 4];
                }
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int32_t pos = pos0 + own_row + k * kAtOnce;
                    if (pos < r.x || pos >= r.y) continue;
                    const float step = __uint_as_float(scale[v][k] << 16), low = __uint_as_float(scale[v][k] & 0xFFFF0000u);
                    T* out = static_cast<T*>(v ? a.v_cache : a.k_cache) + (dst + k * kAtOnce) * D + own * 16;
                    write_eight(out, codes[v][k].x, step, low);
                    write_eight(out + 8, codes[v][k].y, step, low);
                }
        }
        base += total;
        __syncthreads();                                     // before the next chunk rewrites the shared arrays
    }
}

template <typename T, int D>
cudaError_t launch_unpack_t(const CacheUnpackQ4Launch& p, cudaStream_t s) {
    const int64_t cap = (int64_t)(p.a.table_stride < p.a.to_stride ? p.a.table_stride : p.a.to_stride) * p.a.cache.block_size;
    const int64_t items = (cap + kRows - 1) / kRows * p.a.n_seqs * p.a.n_kv_heads, blocks = (items + kWarps - 1) / kWarps;
    note_launch();
    return launch_overlapped(unpack_q4_kernel<T, D>, dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_append_q4(const CacheAppendQ4Launch& p, cudaStream_t s) {
    const int32_t fit = kThreads * kAppendVecs / (2 * p.a.n_kv_heads * (p.a.d / 8));
    const int32_t block_tokens = fit > 1 && p.a.n_tokens > 2 * 152 * (int64_t)fit ? fit : 1;
    const dim3 grid((unsigned)((p.a.n_tokens + block_tokens - 1) / block_tokens));
    note_launch();
    return p.a.dtype == KDA_BF16 ? launch_overlapped(append_q4_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, p, block_tokens)
                                 : launch_overlapped(append_q4_kernel<float>, grid, dim3(kThreads), 0, s, p, block_tokens);
}

cudaError_t launch_unpack_q4(const CacheUnpackQ4Launch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16) return p.a.d == 128 ? launch_unpack_t<__nv_bfloat16, 128>(p, s) : launch_unpack_t<__nv_bfloat16, 64>(p, s);
    return p.a.d == 128 ? launch_unpack_t<float, 128>(p, s) : launch_unpack_t<float, 64>(p, s);
}

}  // namespace kda
